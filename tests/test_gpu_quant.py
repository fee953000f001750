"""The 8-bit chunk pool on the GPU against the 64-bit reference
(tests/quant_reference.py, with the bounds used here): writing and reading
slots, decode attention and chunk mass over codes, and a run of them as a
program would make it."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from oracle import pfd_oracle as orc
from sparse_chunked_kv_gb300 import _abi, api
from sparse_chunked_kv_gb300 import workloads as wl
from tests import parity as P
from tests import quant_reference as R

pytestmark = pytest.mark.gpu

CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
FORMATS = sorted(CODES)
f64 = wl.to_f64


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available()
    _abi.load()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def values_of(pool, name):
    """A pool's values in 64 bits on the host."""
    codes = getattr(pool, name).cpu().to(torch.float64).numpy()
    return R.values(codes, getattr(pool, "exp_" + name).cpu().numpy())


def place(lens, seed=0, gap=0):
    """Slots of these lengths at permuted multiples of 16 rows."""
    order = np.random.RandomState(seed).permutation(len(lens))
    rows, at = [0] * len(lens), 16 * gap
    for j in order:
        rows[j] = at
        at += -(-lens[j] // 16) * 16 + 16 * gap
    return rows, max(at, 16)


def draw_rows(kind, n, hkv, d, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, hkv, d, generator=g)
    if kind == "channels":
        x *= torch.exp(torch.randn(1, hkv, d, generator=g))
    elif kind == "wide":      # every binade of bf16, zeros and subnormals among them
        x = torch.sign(x) * 2.0 ** (torch.rand(n, hkv, d, generator=g) * 250 - 125)
        x[torch.rand(n, hkv, d, generator=g) < 0.1] = 0.0
        x[torch.rand(n, hkv, d, generator=g) < 0.05] = 1e-40
    elif kind == "ties":      # halfway between two codes at scale 1, under a maximum that fixes it
        x = torch.randint(-255, 256, (n, hkv, d), generator=g).float() / 2
        x[:, :, 0] = 127.0
    elif kind == "edges":     # maxima just at and past a power of two times the largest code
        top = torch.tensor([448.0, 450.0, 127.0, 127.5, 1.75, 1.7578125, 1.984375, 1.9921875, 0.0,
                            2.0 ** -92, 2.0 ** -110, 2.0 ** 120])
        x = x.clamp(-1, 1) * top[torch.arange(n) // 16 % len(top)][:, None, None]
        x[:, :, 1] = top[torch.arange(n) // 16 % len(top)][:, None]
    return x.to(torch.bfloat16)


LENS = [1, 15, 16, 17, 0, 129, 64, 33, 200]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("hkv,d", [(1, 64), (2, 128), (5, 64), (4, 128)])
@pytest.mark.parametrize("kind", ["normal", "channels", "wide", "ties", "edges"])
def test_quantize_and_read_back(fmt, hkv, d, kind):
    """Codes, exponents and table are the reference's bit for bit, other pool
    rows keep what they held, and reading back gives code * scale exactly."""
    lens = LENS
    starts = [3 + sum(lens[:j]) + j for j in range(len(lens))]
    n_src = starts[-1] + lens[-1] + 2
    x = {"k": draw_rows(kind, n_src, hkv, d, 1), "v": draw_rows(kind, n_src, hkv, d, 2)}
    rows, pool_rows = place(lens, gap=1)
    pool = api.QuantPool.zeros(pool_rows, hkv, d, CODES[fmt])
    for t in (pool.k, pool.v):
        t.view(torch.uint8).fill_(0x15)
    for t in (pool.exp_k, pool.exp_v):
        t.fill_(99)
    err = ints([0])
    src = ints([[a, n] for a, n in zip(starts, lens)])
    # a wrong bound of the lengths only changes the launch
    for bound in (200, 16):
        table = api.pool_quantize(P.cuda(x["k"]), P.cuda(x["v"]), src, pool, ints(rows),
                                  max_len=bound, dev_err=err)
        assert int(err.item()) == 0
        assert table.cpu().tolist() == [[r, n] for r, n in zip(rows, lens)]
        for name in "kv":
            codes, exps, written = R.quantize(f64(x[name]), lens, starts, rows, pool_rows, fmt)
            got = getattr(pool, name).cpu()
            assert np.array_equal(got.to(torch.float64).numpy()[written], codes[written]), name
            assert (got.view(torch.uint8).numpy()[~written] == 0x15).all(), name
            got = getattr(pool, "exp_" + name).cpu().numpy()
            assert np.array_equal(np.where(exps < 0, 99, exps), got), name
    # back, in another order, one slot twice
    sel = [5, 0, 8, 5, 3, 4, 7]
    at = np.cumsum([1] + [lens[c] + 1 for c in sel])
    k = torch.full((int(at[-1]) + 3, hkv, d), 7.0, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    _, _, dst_table = api.pool_dequantize(pool, table, ints(at[:-1].tolist()), k=k, v=v,
                                          sel=ints(sel), max_len=40, dev_err=err)
    assert int(err.item()) == 0
    assert dst_table.cpu().tolist() == [[int(a), lens[c]] for a, c in zip(at, sel)]
    for name, got in (("k", k), ("v", v)):
        want = np.full(tuple(got.shape), 7.0)
        vals = values_of(pool, name)
        for a, c in zip(at, sel):
            want[a:a + lens[c]] = vals[rows[c]:rows[c] + lens[c]]
        assert np.array_equal(got.cpu().to(torch.float64).numpy(), want), name


@pytest.mark.parametrize("fmt", FORMATS)
def test_non_finite_blocks(fmt):
    """A NaN or an infinity marks its own (block, head) and no other."""
    x = draw_rows("normal", 48, 2, 64, 5)
    x[3, 0, 9], x[20, 1, 0], x[21, 1, 5] = math.inf, math.nan, -math.inf
    pool = api.QuantPool.zeros(48, 2, 64, CODES[fmt])
    table = api.pool_quantize(P.cuda(x), P.cuda(x), ints([[0, 48]]), pool, ints([0]))
    assert (pool.exp_k.cpu() == 255).tolist() == [[True, False], [False, True], [False, False]]
    k, v, _ = api.pool_dequantize(pool, table, ints([0]), 48)
    bad = torch.isnan(k.cpu()).all(dim=2)
    assert bad[:16, 0].all() and bad[16:32, 1].all() and int(bad.sum()) == 32
    assert int(torch.isnan(k).sum()) == 32 * 64 and torch.equal(torch.isnan(k), torch.isnan(v))


def test_slot_errors_are_reported_and_skipped():
    x = P.cuda(draw_rows("normal", 64, 2, 64, 5))
    pool = api.QuantPool.zeros(64, 2, 64)

    def write(src, row):
        err = ints([0])
        before = pool.k.view(torch.uint8).clone()
        table = api.pool_quantize(x, x, ints([src]), pool, ints([row]), max_len=64, dev_err=err)
        same = torch.equal(before, pool.k.view(torch.uint8))
        return int(err.item()), table.cpu().tolist()[0], same

    assert write([-1, 4], 0) == (_abi.DEVERR_TABLE, [0, 0], True)
    assert write([0, -4], 0) == (_abi.DEVERR_TABLE, [0, 0], True)
    assert write([61, 4], 0) == (_abi.DEVERR_TABLE, [0, 0], True)
    assert write([2 ** 31 - 1, 2 ** 31 - 1], 0) == (_abi.DEVERR_TABLE, [0, 0], True)
    assert write([0, 4], 8) == (_abi.DEVERR_SLOT, [0, 0], True)
    assert write([0, 4], -16) == (_abi.DEVERR_SLOT, [0, 0], True)
    assert write([0, 17], 48) == (_abi.DEVERR_SLOT, [0, 0], True)
    assert write([0, 4], 2 ** 31 - 16) == (_abi.DEVERR_SLOT, [0, 0], True)
    assert write([0, 16], 48) == (0, [48, 16], False)

    def read(entry, sel, row):
        err = ints([0])
        k = torch.full((64, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        _, _, table = api.pool_dequantize(pool, ints([entry]), ints([row]), k=k, v=k.clone(),
                                          sel=ints([sel]), max_len=64, dev_err=err)
        return int(err.item()), table.cpu().tolist()[0], bool((k == 7.0).all())

    assert read([0, 16], 1, 0) == (_abi.DEVERR_SEL, [0, 0], True)
    assert read([0, 16], -1, 0) == (_abi.DEVERR_SEL, [0, 0], True)
    assert read([8, 16], 0, 0) == (_abi.DEVERR_TABLE, [0, 0], True)
    assert read([48, 17], 0, 0) == (_abi.DEVERR_TABLE, [0, 0], True)
    assert read([48, 16], 0, 49) == (_abi.DEVERR_SLOT, [0, 0], True)
    assert read([48, 16], 0, 48) == (0, [48, 16], False)


def test_reading_back_into_no_rows():
    """Slots without a destination row are refused, empty ones too; no slots need
    none, and empty slots with a row get their entries."""
    pool = api.QuantPool.zeros(64, 2, 64)
    for entry in ([0, 0], [0, 5]):
        with pytest.raises(ValueError, match="dst_rows"):
            api.pool_dequantize(pool, ints([entry]), ints([0]), 0)
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="dst_rows"):
        api.pool_dequantize(pool, ints([[0, 0]]), ints([0]), k=none, v=none)
    k, v, table = api.pool_dequantize(pool, torch.empty(0, 2, dtype=torch.int32, device="cuda"),
                                      torch.empty(0, dtype=torch.int32, device="cuda"), 0)
    assert k.shape == v.shape == (0, 2, 64) and table.shape == (0, 2)
    given, err = ints([[7, 7], [7, 7], [7, 7]]), ints([0])
    api.pool_dequantize(pool, ints([[0, 0], [16, 0], [32, 2]]), ints([0, 1, 1]), 1, dst_table=given, dev_err=err)
    assert given.tolist() == [[0, 0], [1, 0], [0, 0]] and int(err.item()) == _abi.DEVERR_SLOT


# ---------------------------------------------------------------- decode --

class Step:
    """One decode step over a quantised pool, with its 64-bit reference."""

    def __init__(self, fmt, hq, hkv, d, lqs, chunk_lens, self_keys=True, seed=0, spare=3,
                 kind="channels", q_scale=1.0):
        self.fmt, self.hq, self.hkv, self.d, self.self_keys = fmt, hq, hkv, d, self_keys
        rng = np.random.RandomState(seed)
        flat = [n for c in chunk_lens for n in c]
        lens = flat + [37] * spare
        perm = rng.permutation(len(lens)).tolist()      # table order
        self.lens = [0] * len(lens)
        for i, at in enumerate(perm):
            self.lens[at] = lens[i]
        self.sel_host = perm[:len(flat)]
        rows, pool_rows = place(self.lens, seed)
        starts = np.cumsum([0] + self.lens).tolist()
        k, v = draw_rows(kind, max(starts[-1], 1), hkv, d, seed + 1), draw_rows("normal", max(starts[-1], 1), hkv, d, seed + 2)
        self.pool = api.QuantPool.zeros(pool_rows, hkv, d, CODES[fmt])
        # rows that no slot covers hold codes and exponents that would show
        for t in (self.pool.k, self.pool.v):
            t.view(torch.uint8).fill_(0x7F)
        for t in (self.pool.exp_k, self.pool.exp_v):
            t.fill_(255)
        self.table = api.pool_quantize(P.cuda(k), P.cuda(v),
                                       ints([[a, n] for a, n in zip(starts, self.lens)]), self.pool,
                                       ints(rows))
        self.sel = ints(self.sel_host)
        self.cu_lq = np.cumsum([0] + list(lqs)).tolist()
        self.cu_k = np.cumsum([0] + [len(c) for c in chunk_lens]).tolist()
        total = self.cu_lq[-1]
        g = torch.Generator().manual_seed(seed + 3)
        self.q = (q_scale * torch.randn(total, hq, d, generator=g)).to(torch.bfloat16)
        self.k_self, self.v_self = draw_rows(kind, total, hkv, d, seed + 4), draw_rows("normal", total, hkv, d, seed + 5)
        self.max_len = max(self.lens + [1])

    def run(self, n_splits=0, **kw):
        plan = api.QuantDecodePlan(self.cu_lq, self.cu_k, self.hq, self.hkv, self.d, self.max_len,
                                   self_keys=self.self_keys, n_splits=n_splits)
        err = ints([0])
        if self.self_keys:
            out, lse = api.decode_attention_quant(P.cuda(self.q), P.cuda(self.k_self),
                                                  P.cuda(self.v_self), self.pool, self.table,
                                                  self.sel, plan, dev_err=err, **kw)
        else:
            out, lse = api.decode_partial_quant(P.cuda(self.q), None, None, self.pool, self.table,
                                                self.sel, plan, dev_err=err, **kw)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        return out, lse

    def reference(self):
        pk, pv = values_of(self.pool, "k"), values_of(self.pool, "v")
        table = self.table.cpu().numpy()
        parts = []
        for b in range(len(self.cu_lq) - 1):
            a, z = self.cu_lq[b], self.cu_lq[b + 1]
            chunks = self.sel_host[self.cu_k[b]:self.cu_k[b + 1]]
            keys, vals = R.keys_of(pk, table, chunks), R.keys_of(pv, table, chunks)
            if self.self_keys:
                keys = np.concatenate([keys, f64(self.k_self[a:z])])
                vals = np.concatenate([vals, f64(self.v_self[a:z])])
            parts.append(R.decode(f64(self.q[a:z]), keys, vals, 1 / math.sqrt(self.d)))
        return [np.concatenate(p) for p in zip(*parts)]

    def check(self, out, lse, ref=None):
        want, want_lse, tol, lse_tol = ref or self.reference()
        got, got_lse = out.cpu().to(torch.float64).numpy(), lse.cpu().to(torch.float64).numpy()
        empty = np.isneginf(want_lse)
        assert np.array_equal(np.isneginf(got_lse), empty)
        assert (got[empty] == 0).all()
        off = np.abs(got - want)
        assert (off <= tol).all(), f"out: {off.max():.3e}, {(off / np.maximum(tol, 1e-30)).max():.2f} of its bound"
        off = np.abs(got_lse[~empty] - want_lse[~empty])
        assert (off <= lse_tol[~empty]).all(), f"lse: {off.max():.3e}"


DECODE = {
    # one token: over one row, over nothing but itself, over ragged chunks
    "one_row": dict(hq=8, hkv=2, d=64, lqs=[1], chunk_lens=[[1]]),
    "no_chunks": dict(hq=8, hkv=2, d=64, lqs=[1], chunk_lens=[[]]),
    "token": dict(hq=28, hkv=4, d=128, lqs=[1], chunk_lens=[[1, 15, 16, 17, 0, 129, 255]]),
    "token_mha": dict(hq=4, hkv=4, d=64, lqs=[1], chunk_lens=[[130, 7]]),
    "token_mqa": dict(hq=128, hkv=1, d=128, lqs=[1], chunk_lens=[[130, 7]]),
    # a ragged batch, a sequence without rows and one without chunks among it
    "batch": dict(hq=8, hkv=2, d=64, lqs=[3, 0, 1, 20], chunk_lens=[[40, 3], [9], [], [16, 16, 100]]),
    "drafts": dict(hq=28, hkv=4, d=128, lqs=[1, 9, 4], chunk_lens=[[300, 200], [77, 129, 1], [64]]),
    # live rows of several query tiles
    "rows": dict(hq=28, hkv=4, d=128, lqs=[50], chunk_lens=[[129, 65, 257]]),
    "rows_mha": dict(hq=2, hkv=2, d=128, lqs=[300], chunk_lens=[[100, 33]]),
    "rows_odd": dict(hq=10, hkv=2, d=64, lqs=[77, 30], chunk_lens=[[31, 2, 2, 2, 90], [500]]),
    "long": dict(hq=4, hkv=1, d=64, lqs=[2], chunk_lens=[[2049] * 8]),
    # one query tile a sequence (two splits a CTA): full, ragged, of unlike lengths
    "tile": dict(hq=28, hkv=4, d=128, lqs=[18], chunk_lens=[[129] * 9]),
    "tiles": dict(hq=8, hkv=2, d=64, lqs=[9, 31, 1, 0, 32], chunk_lens=[[700, 3], [17], [], [5], [1] * 20]),
    # enough rows and keys that the chunks are read back to bf16 first
    "staged": dict(hq=8, hkv=2, d=64, lqs=[200, 65], chunk_lens=[[2049] * 8, [300, 0, 2049, 1]]),
}


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("self_keys", [True, False])
@pytest.mark.parametrize("name", sorted(DECODE))
def test_decode_matches_the_reference(name, self_keys, fmt):
    st = Step(fmt, self_keys=self_keys, seed=len(name), **DECODE[name])
    ref = st.reference()
    for n_splits in (0, 1, 2, 10, 3):
        out, lse = st.run(n_splits)
        st.check(out, lse, ref)
    again, lse2 = st.run(3)
    assert torch.equal(again, out) and torch.equal(lse2, lse), "repeated calls give the same bits"


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_scale", [0.0, 30.0])
def test_decode_flat_and_peaked(fmt, q_scale):
    """All keys alike, and one key that takes nearly everything."""
    st = Step(fmt, 8, 2, 64, [5], [[200, 31]], seed=3, q_scale=q_scale)
    st.check(*st.run())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lq,longest", [(1, 128), (8, 128), (20, 128), (32, 128), (40, 128), (200, 2048)])
def test_decode_rising_logits(lq, longest, fmt):
    """Every few tiles of keys pass the maximum so far by far, by each of the ways
    a step may run: what was summed before is rescaled."""
    st = Step(fmt, 8, 2, 64, [lq], [[longest] * 10], seed=21, self_keys=False)
    st.q = st.q.abs()
    codes = st.pool.k.view(torch.uint8)
    if fmt == "e4m3":
        codes &= 0x7F
        codes[codes == 0x7F] = 0
    else:
        st.pool.k.copy_(st.pool.k.to(torch.int16).abs().clamp(max=127).to(torch.int8))
    for j, c in enumerate(st.sel_host):
        row = int(st.table[c, 0].item()) // 16
        st.pool.exp_k[row:row + longest // 16] += j - 4 if j > 4 else 0
    ref = st.reference()
    for n_splits in (1, 2):
        st.check(*st.run(n_splits), ref)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lq", [1, 20, 40])
def test_decode_scales_far_from_one(fmt, lq):
    """Exponents from 2^-60 to 2^60 in one step: a key that large decides its
    rows alone, and values of any size are read exactly."""
    st = Step(fmt, 8, 2, 64, [lq], [[64, 48, 31]], seed=4)
    for j, (row, n) in enumerate(st.table.cpu().tolist()):
        b = slice(row // 16, row // 16 + -(-n // 16))
        st.pool.exp_v[b] = 127 + (60 if j % 2 else -60)
        st.pool.exp_k[b] = 127 - 60 if j % 2 else 127
    st.check(*st.run())


@pytest.mark.parametrize("lq,more", [(1, 0), (20, 0), (40, 0), (200, 8)])
@pytest.mark.parametrize("fmt,byte", [("int8", 0), ("int8", 1), ("int8", 9), ("e4m3", 3), ("e4m3", 9)])
def test_scales_at_the_low_end(fmt, byte, lq, more):
    """Scales down to 2^-127, smaller than any that quantising writes, by each of the
    ways a step may run and in a mass: every value is exact in bf16 down to
    2^-133 (E4M3 codes are multiples of 2^-9, so from byte 3 on)."""
    st = Step(fmt, 8, 2, 64, [lq], [[64, 40] + [2049] * more], seed=42, self_keys=False, spare=0)
    st.pool.exp_v.fill_(byte)
    ref = st.reference()
    for n_splits in (1, 3):
        st.check(*st.run(n_splits), ref)
    st.pool.exp_v.fill_(127)
    st.pool.exp_k.fill_(byte)
    st.q = (st.q.float() * 2.0 ** (120 - byte)).to(torch.bfloat16)   # the logits of scale 2^-7
    ref = st.reference()
    for n_splits in (1, 3):
        out, lse = st.run(n_splits)
        st.check(out, lse, ref)
    n = st.table.shape[0]
    got = api.chunk_mass_quant(P.cuda(st.q), st.pool, st.table, lse,
                               api.QuantMassPlan([0, lq], [0, n], 8, 2, 64))
    want, tol = R.mass(f64(st.q), values_of(st.pool, "k"), st.table.cpu().numpy(), range(n),
                       f64(lse.cpu()), 1 / 8)
    assert (np.abs(got.cpu().to(torch.float64).numpy() - want) <= tol).all()


@pytest.mark.parametrize("byte", [0, 1, 2])
def test_scales_at_the_low_end_few_rows(byte):
    """The few-rows kernel takes codes in f16 and scales in fp32: exact from byte 0 on."""
    st = Step("e4m3", 8, 2, 64, [3], [[64, 40]], seed=43, self_keys=False, spare=0)
    st.pool.exp_v.fill_(byte)
    for n_splits in (1, 3):
        st.check(*st.run(n_splits))
    st.pool.exp_v.fill_(127)
    st.pool.exp_k.fill_(byte)
    st.q = (st.q.float() * 2.0 ** (120 - byte)).to(torch.bfloat16)
    for n_splits in (1, 3):
        st.check(*st.run(n_splits))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lq", [40, 320])
def test_decode_equals_decode_over_the_values(fmt, d, lq):
    """Over slots of whole blocks one split gives the bits of
    pfd_decode_attention over the dequantised pool: the same products in the
    same order, as every value is exact in bf16."""
    st = Step(fmt, 28, 4, d, [lq], [[256, 16, 48, 128]], seed=6, spare=0)
    out, lse = st.run(1)
    rows = st.table[:, 0].contiguous()
    k, v, table = api.pool_dequantize(st.pool, st.table, rows, st.pool.rows)
    want, want_lse = api.decode_attention(P.cuda(st.q), P.cuda(st.k_self), P.cuda(st.v_self), k, v,
                                          table, st.sel, n_splits=1)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("lq", [1, 20, 40])
def test_decode_nan_block_shows(lq):
    """A block marked NaN makes its head's rows NaN and leaves other heads alone."""
    st = Step("e4m3", 8, 2, 64, [lq], [[64, 40]], seed=8)
    out, _ = st.run()
    row = st.table.cpu().tolist()[st.sel_host[1]][0]
    st.pool.exp_v[row // 16, 1] = 255
    bad, _ = st.run()
    assert torch.isnan(bad[:, 4:]).all() and torch.equal(bad[:, :4], out[:, :4])
    # a whole split's keys
    st = Step("e4m3", 8, 2, 64, [lq], [[256] * 4], self_keys=False, seed=8)
    st.pool.exp_k[st.table.cpu().tolist()[st.sel_host[1]][0] // 16:][:16, 1] = 255
    for n_splits in (1, 4, 8):
        bad, lse = st.run(n_splits)
        assert torch.isnan(bad[:, 4:]).all() and torch.isnan(lse[:, 4:]).all()
        assert torch.isfinite(bad[:, :4]).all() and torch.isfinite(lse[:, :4]).all()


@pytest.mark.parametrize("lq,more", [(1, 0), (20, 0), (40, 0), (200, 8)])
def test_decode_bad_table_and_selection(lq, more):
    """Misplaced entries and selections are reported and skipped, by each of
    the ways a step may run."""
    st = Step("int8", 8, 2, 64, [lq], [[64, 40, 17] + [2049] * more], seed=9)
    plan = api.QuantDecodePlan(st.cu_lq, st.cu_k, 8, 2, 64, st.max_len)
    good = st.table.clone()

    def run(table, sel):
        err = ints([0])
        out, lse = api.decode_attention_quant(P.cuda(st.q), P.cuda(st.k_self), P.cuda(st.v_self),
                                              st.pool, table, sel, plan, dev_err=err)
        torch.cuda.synchronize()
        return int(err.item()), out, lse

    # the same step with the second chunk's place in the selection left out
    table = good.clone()
    table[st.sel_host[1], 1] = 0
    _, want, want_lse = run(table, st.sel)
    # (a slot of one row more than the plan's bound among them)
    for entry in ([8, 40], [-16, 40], [0, -1], [st.pool.rows, 16], [st.pool.rows - 16, 17],
                  [2 ** 31 - 16, 2 ** 31 - 1], [0, st.max_len + 1]):
        table = good.clone()
        table[st.sel_host[1]] = ints(entry)
        err, out, lse = run(table, st.sel)
        assert err == _abi.DEVERR_TABLE and torch.equal(out, want) and torch.equal(lse, want_lse), entry
    for index in (-1, good.shape[0], 2 ** 31 - 1):
        sel = st.sel.clone()
        sel[1] = index
        err, out, lse = run(good, sel)
        assert err == _abi.DEVERR_SEL and torch.equal(out, want) and torch.equal(lse, want_lse), index


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lq,more", [(1, 0), (20, 0), (40, 0), (200, 8)])
def test_decode_chunk_selected_twice(lq, more, fmt):
    """A chunk that is selected twice counts twice."""
    st = Step(fmt, 8, 2, 64, [lq, 1], [[64, 40, 17] + [2049] * more, [33, 2]], seed=10)
    st.sel_host[1], st.sel_host[3 + more] = st.sel_host[0], st.sel_host[4 + more]
    st.sel = ints(st.sel_host)
    st.check(*st.run())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("hq,hkv,d,lq", [(16, 16, 64, 2), (10, 5, 128, 3), (128, 1, 128, 2), (21, 3, 64, 30)])
def test_decode_most_chunks_and_heads(hq, hkv, d, lq, fmt):
    """511 chunks of a sequence, the most, and odd numbers of heads."""
    st = Step(fmt, hq, hkv, d, [lq], [[1, 16, 5] * 170 + [18]], seed=14, spare=0)
    ref = st.reference()
    for n_splits in (0, 64):
        st.check(*st.run(n_splits), ref)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("batch", [7, 64, 65])
@pytest.mark.parametrize("lq", [2, 12, 70])
def test_decode_ragged_batch(batch, lq, fmt):
    """Sequences of very different numbers of keys and rows, none among them,
    over one workspace whose former contents would show."""
    rng = np.random.RandomState(batch + lq)
    lqs = [int(x) for x in rng.randint(0, lq + 1, batch)]
    lqs[batch // 2] = lq
    chunk_lens = [[int(x) for x in rng.randint(0, 60, rng.randint(0, 5))] for _ in range(batch)]
    chunk_lens[batch // 3], chunk_lens[batch // 2] = [60] * 30, [60, 0, 60] * 7
    st = Step(fmt, 8, 2, 64, lqs, chunk_lens, seed=20, self_keys=lq != 12)
    ref = st.reference()
    for n_splits in (0, 5, 64):
        plan = api.QuantDecodePlan(st.cu_lq, st.cu_k, 8, 2, 64, st.max_len, self_keys=st.self_keys,
                                   n_splits=n_splits)
        ws = torch.full((max(plan.workspace_bytes, 1),), 0x7F, dtype=torch.uint8, device="cuda")
        ws.view(torch.uint8)[1::4] = 0x00
        st.check(*st.run(n_splits, workspace=ws), ref)


@pytest.mark.parametrize("lq,more", [(3, 0), (20, 0), (40, 0), (200, 8)])
def test_decode_non_finite_live_rows(lq, more):
    """An infinity or NaN among the live rows reaches what it is a factor of,
    and nothing beside it: a value its own column, a logit of -inf no output, a
    query row its own outputs."""
    st = Step("e4m3", 8, 2, 64, [lq], [[64, 40, 17] + [2049] * more], seed=15)
    st.q[:, :, 7] = st.q[:, :, 7].abs() + 0.5
    st.k_self[2, :, 7] = 0.0
    clean = st.reference()
    k, v, q = st.k_self.clone(), st.v_self.clone(), st.q.clone()
    # the third live key at logit -inf: the reference leaves it out
    st.k_self[2, :, 7] = -math.inf
    keys, vals = (np.concatenate([R.keys_of(values_of(st.pool, x), st.table.cpu().numpy(), st.sel_host),
                                  np.delete(f64(y), 2, axis=0)]) for x, y in zip("kv", (k, v)))
    st.check(*st.run(), R.decode(f64(q), keys, vals, 1 / 8))
    st.k_self = k
    # values: one column of the first KV head
    for bad in (math.inf, math.nan):
        st.v_self = v.clone()
        st.v_self[1, 0, 5] = bad
        out, lse = st.run()
        hit = torch.zeros(out.shape, dtype=torch.bool)
        hit[:, :4, 5] = True
        host = out.cpu()
        assert not torch.isfinite(host[hit]).any()
        host[hit] = torch.from_numpy(clean[0])[hit].to(host.dtype)
        st.check(host, lse, clean)
    st.v_self = v
    # a query row
    st.q = q.clone()
    st.q[1, 3, 9] = math.nan
    for n_splits in (1, 3, 9):
        out, lse = (x.cpu() for x in st.run(n_splits))
        assert torch.isnan(out[1, 3]).all() and torch.isnan(lse[1, 3])
        out[1, 3], lse[1, 3] = torch.from_numpy(clean[0][1, 3]).to(out.dtype), float(clean[1][1, 3])
        st.check(out, lse, clean)


MINUS_INF = {
    # live rows, chunks, and a number of splits that leaves one with live keys alone
    "rows": (5, [[64, 128]], 13),
    "tile": (30, [[64, 128]], 14),
    "tiles": (40, [[64, 128]], 15),
    "staged": (352, [[2049] * 8], 64),
}


def _at_minus_inf(st, keys):
    """Gives these live keys (a slice) logits of -inf from every query."""
    st.q[:, :, 7] = st.q[:, :, 7].abs() + 0.5
    st.k_self[keys, :, 7] = -math.inf


@pytest.mark.parametrize("name", sorted(MINUS_INF))
def test_split_with_logits_of_minus_infinity_only(name):
    """Live keys at logit -inf count for nothing, also where a split holds no
    others, by each of the ways a step may run and over the bf16 pool."""
    lq, chunk_lens, n_splits = MINUS_INF[name]
    st = Step("e4m3", 8, 2, 64, [lq], chunk_lens, seed=40)
    _at_minus_inf(st, slice(None))
    host = st.table.cpu().numpy()
    keys, vals = (R.keys_of(values_of(st.pool, x), host, st.sel_host) for x in "kv")
    ref = R.decode(f64(st.q), keys, vals, 1 / 8)
    k, v, table = api.pool_dequantize(st.pool, st.table, st.table[:, 0].contiguous(), st.pool.rows)
    # The bf16 pool's splits keep their outputs in bf16: half a step of each, so of
    # their weighed sum, 2^-8 A at most; the bound without it is 2^-8 A at least.
    ref2 = (ref[0], ref[1], 2 * ref[2], ref[3])
    for n in (0, 1, n_splits):
        st.check(*st.run(n), ref)
        out, lse = api.decode_attention(P.cuda(st.q), P.cuda(st.k_self), P.cuda(st.v_self), k, v,
                                        table, st.sel, n_splits=n)
        st.check(out, lse, ref2)


@pytest.mark.parametrize("lq", [3, 20, 32, 40, 200])
@pytest.mark.parametrize("first", [16, 64, 128, 200])
def test_first_logits_of_minus_infinity(lq, first):
    """The first keys of a row at logit -inf, up to all of them: the others
    decide, and a row with no other gives 0 and -inf."""
    st = Step("e4m3", 8, 2, 64, [lq], [[]], seed=41)
    cut = min(first, lq)
    _at_minus_inf(st, slice(0, cut))
    ref = R.decode(f64(st.q), f64(st.k_self[cut:]), f64(st.v_self[cut:]), 1 / 8)
    ref2 = (ref[0], ref[1], 2 * ref[2], ref[3])
    for n in (1, 2, 64):
        st.check(*st.run(n), ref)
        out, lse = api.decode_attention(P.cuda(st.q), P.cuda(st.k_self), P.cuda(st.v_self), st.pool.k[:0].bfloat16(),
                                        st.pool.v[:0].bfloat16(), st.table[:0], st.sel, n_splits=n)
        st.check(out, lse, ref2)


def test_nan_shows_through_bf16_splits():
    """The bf16 pool's calls: a split whose keys are all NaN, and a NaN among a
    split's others, reach their head's rows and no others'."""
    st = Step("e4m3", 8, 2, 64, [40], [[256] * 4], seed=8)
    k, v, table = api.pool_dequantize(st.pool, st.table, st.table[:, 0].contiguous(), st.pool.rows)
    row = st.table.cpu().tolist()[st.sel_host[1]][0]
    for rows in (slice(row, row + 256), slice(row + 9, row + 10)):
        bad = k.clone()
        bad[rows, 1] = math.nan
        for n in (1, 4, 8):
            out, lse = api.decode_attention(P.cuda(st.q), P.cuda(st.k_self), P.cuda(st.v_self), bad, v,
                                            table, st.sel, n_splits=n)
            assert torch.isnan(out[:, 4:]).all() and torch.isnan(lse[:, 4:]).all()
            assert torch.isfinite(out[:, :4]).all() and torch.isfinite(lse[:, :4]).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("self_keys", [True, False])
@pytest.mark.parametrize("hq,hkv,d,lqs,chunk_lens", [
    (16, 16, 64, [32], [[2049, 129]]), (16, 16, 64, [17, 3, 20], [[900], [], [2049, 0, 16, 200]]),
    (28, 4, 64, [4], [[2049] * 4 + [513]]), (16, 16, 128, [20], [[2049] * 4 + [129]]),
    (64, 16, 128, [8, 1], [[2049] * 4, [130, 7]])])
def test_long_steps_of_17_to_32_rows(hq, hkv, d, lqs, chunk_lens, self_keys, fmt):
    """So many keys that the few-rows kernel takes them, with four tiles of rows."""
    st = Step(fmt, hq, hkv, d, lqs, chunk_lens, self_keys=self_keys, seed=45)
    groups = sum(-(-st.max_len // 16) * len(c) for c in chunk_lens) * hkv
    assert groups >= (14 if d == 64 else 55) * torch.cuda.get_device_properties(0).multi_processor_count
    ref = st.reference()
    for n_splits in (0, 1, 3, 64):
        st.check(*st.run(n_splits), ref)
    again, lse = st.run(3)
    st.check(again, lse, ref)


@pytest.mark.parametrize("lq", [17, 32])
def test_long_steps_of_17_to_32_rows_at_the_edges(lq):
    """Rising logits, and live keys at -inf, NaN and infinity."""
    st = Step("e4m3", 16, 16, 64, [lq], [[128] * 18], seed=46)
    st.q = st.q.abs()
    st.pool.k.view(torch.uint8).bitwise_and_(0x7F)
    st.pool.k.view(torch.uint8)[st.pool.k.view(torch.uint8) == 0x7F] = 0
    for j, c in enumerate(st.sel_host):
        row = int(st.table[c, 0].item()) // 16
        st.pool.exp_k[row:row + 8] += max(0, (j - 8) // 2)
    st.k_self[:, :, 7] = -math.inf
    st.q[:, :, 7] += 0.5
    host = st.table.cpu().numpy()
    keys, vals = (R.keys_of(values_of(st.pool, x), host, st.sel_host) for x in "kv")
    ref = R.decode(f64(st.q), keys, vals, 1 / 8)
    for n in (1, 2, 64):
        st.check(*st.run(n), ref)
    st.k_self = draw_rows("normal", lq, 16, 64, 1)
    clean = st.reference()
    st.q[1, 3, 9] = math.nan
    for n in (1, 3):
        out, lse = (x.cpu() for x in st.run(n))
        assert torch.isnan(out[1, 3]).all() and torch.isnan(lse[1, 3])
        out[1, 3], lse[1, 3] = torch.from_numpy(clean[0][1, 3]).to(out.dtype), float(clean[1][1, 3])
        st.check(out, lse, clean)


def _assert_staged(st):
    """The step's chunks are read back to bf16 first (its workspace holds the copy)."""
    need = _abi.pfd_decode_quant_workspace(len(st.cu_lq) - 1, st.cu_lq, st.cu_k, st.hq, st.hkv, st.d,
                                           st.max_len, int(st.self_keys), 1)
    assert need >= st.cu_k[-1] * st.max_len * 4 * st.hkv * st.d


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("self_keys", [True, False])
@pytest.mark.parametrize("d,lqs", [(64, [352, 65]), (128, [400, 65])])
def test_staged_steps_match_the_reference(d, lqs, self_keys, fmt):
    """Enough rows and keys that the chunks are read back first: a ragged batch."""
    st = Step(fmt, 8, 2, d, lqs, [[2049] * 8, [300, 0, 2049, 1]], self_keys=self_keys, seed=44)
    _assert_staged(st)
    ref = st.reference()
    for n_splits in (0, 1, 3, 64):
        st.check(*st.run(n_splits), ref)


@pytest.mark.parametrize("check", [
    lambda: test_decode_bad_table_and_selection(352, 8),
    lambda: test_decode_chunk_selected_twice(352, 8, "int8"),
    lambda: test_decode_non_finite_live_rows(352, 8),
    lambda: test_two_graphs_in_turn(352, 8),
    lambda: test_scales_at_the_low_end("e4m3", 3, 352, 8)],
    ids=["bad_entries", "twice", "non_finite", "graphs", "low_end"])
def test_staged_steps_at_the_edges(check):
    _assert_staged(Step("int8", 8, 2, 64, [352], [[64, 40, 17] + [2049] * 8]))
    _assert_staged(Step("int8", 8, 2, 64, [352], [[64, 40] + [2049] * 8]))
    check()


def test_steps_without_rows_or_chunks():
    """Nothing to compute: outputs of no rows, a mass of zeros, an empty mass."""
    st = Step("int8", 8, 2, 64, [3], [[64, 17]], seed=16)
    pool, table, sel = st.pool, st.table, st.sel
    none = torch.empty(0, 8, 64, dtype=torch.bfloat16, device="cuda")
    kv = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    out, lse = api.decode_attention_quant(none, kv, kv, pool, table, sel,
                                          api.QuantDecodePlan([0, 0, 0], [0, 1, 2], 8, 2, 64, 64))
    assert out.shape == (0, 8, 64) and lse.shape == (0, 8)
    n = table.shape[0]
    mass = api.chunk_mass_quant(none, pool, table, lse, api.QuantMassPlan([0, 0], [0, n], 8, 2, 64))
    assert mass.shape == (n,) and (mass == 0).all()
    q = P.cuda(st.q)
    mass = api.chunk_mass_quant(q, pool, table[:0], torch.zeros(3, 8, device="cuda"),
                                api.QuantMassPlan([0, 3], [0, 0], 8, 2, 64))
    assert mass.shape == (0,)
    # rows over an empty table and their own keys only
    plan = api.QuantDecodePlan([0, 3], [0, 0], 8, 2, 64, 0)
    out, lse = api.decode_attention_quant(q, P.cuda(st.k_self), P.cuda(st.v_self), pool, table[:0],
                                          sel[:0], plan)
    k, v = f64(st.k_self), f64(st.v_self)
    st.check(out, lse, R.decode(f64(st.q), k, v, 1 / 8))


# ------------------------------------------------------------------ mass --

def test_mass_without_a_finite_normaliser():
    """A row whose lse is -inf (no key) or NaN adds nothing to any chunk."""
    st = Step("e4m3", 8, 2, 64, [5], [[100, 31, 16]], seed=17, spare=0)
    q, n = P.cuda(st.q), st.table.shape[0]
    lse = torch.full((5, 8), 3.0, device="cuda")
    plan = api.QuantMassPlan([0, 5], [0, n], 8, 2, 64)
    lse[2, 1], lse[4, 7] = -math.inf, math.nan
    got = api.chunk_mass_quant(q, st.pool, st.table, lse, plan).cpu().to(torch.float64).numpy()
    far = lse.clone()
    far[2, 1] = far[4, 7] = 1e4         # exp(s - 1e4) = 0
    want, tol = R.mass(f64(st.q), values_of(st.pool, "k"), st.table.cpu().numpy(), range(n),
                       f64(far.cpu()), 1 / 8)
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("lens", [[100, 31, 16], [17] * 1100])   # one chunk an item, and several
@pytest.mark.parametrize("lq", [5, 40])
def test_mass_of_a_query_row_that_is_not_finite(lq, lens, bad):
    """A NaN or an infinity in a query row makes its lse NaN; the row adds nothing
    to any chunk, over the 8-bit and the bf16 pool, and the others what they did."""
    st = Step("e4m3", 8, 2, 64, [lq], [lens], seed=17, spare=0)
    st.cu_k, st.sel = [0, 3], st.sel[:3].clone()      # the step selects three chunks
    n = st.table.shape[0]
    st.q[1, 3, 9], st.q[lq - 1, 6, 0] = bad, bad
    q = P.cuda(st.q)
    _, lse = st.run()
    hit = torch.zeros(lq, 8, dtype=torch.bool)
    hit[1, 3] = hit[lq - 1, 6] = True
    assert torch.equal(torch.isnan(lse).cpu(), hit)
    got = api.chunk_mass_quant(q, st.pool, st.table, lse, api.QuantMassPlan([0, lq], [0, n], 8, 2, 64))
    k, _, table = api.pool_dequantize(st.pool, st.table, st.table[:, 0].contiguous(), st.pool.rows)
    mass = torch.full((n,), 7.0, device="cuda")
    need = _abi.pfd_chunk_mass_workspace(1, [0, lq], [0, n], 8, 2)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    _abi.pfd_chunk_mass(q, ints([0, lq]), [0, lq], k, k.shape[0], table, n, [0, n], lse, 1, 8, 2, 64,
                        0.0, mass, None, ws, need)
    x, at = f64(st.q), f64(lse.cpu())
    x[hit.numpy()], at[hit.numpy()] = 0.0, 1e4        # exp(0 - 1e4) = 0
    want, tol = R.mass(x, values_of(st.pool, "k"), st.table.cpu().numpy(), range(n), at, 1 / 8)
    for m in (got, mass):
        assert (np.abs(m.cpu().to(torch.float64).numpy() - want) <= tol).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("case", ["small", "batch", "many", "one"])
def test_mass_matches_the_reference(case, fmt):
    sizes = {
        "small": dict(hq=8, hkv=2, d=64, lqs=[20], chunk_lens=[[100, 31, 16, 1, 0]]),
        "batch": dict(hq=28, hkv=4, d=128, lqs=[9, 0, 40], chunk_lens=[[129] * 3, [20], [65, 257]]),
        "many": dict(hq=4, hkv=2, d=64, lqs=[30], chunk_lens=[[17] * 1100]),
        "one": dict(hq=28, hkv=4, d=128, lqs=[1], chunk_lens=[[300, 129]]),
    }[case]
    st = Step(fmt, seed=11, spare=0, **sizes)
    # the chunks of a mass call are table ranges: lay the table out by sequence
    table = st.table[st.sel.long()].contiguous()
    # the step had selected each sequence's first three chunks
    pk, host = values_of(st.pool, "k"), table.cpu().numpy()
    lse = torch.zeros(st.cu_lq[-1], st.hq)
    for b in range(len(st.cu_lq) - 1):
        a, z, n0, n1 = st.cu_lq[b], st.cu_lq[b + 1], st.cu_k[b], st.cu_k[b + 1]
        keys = np.concatenate([R.keys_of(pk, host, range(n0, min(n0 + 3, n1))), f64(st.k_self[a:z])])
        lse[a:z] = torch.from_numpy(R.decode(f64(st.q[a:z]), keys, keys, 1 / math.sqrt(st.d))[1])
    lse = P.cuda(lse)
    plan = api.QuantMassPlan(st.cu_lq, st.cu_k, st.hq, st.hkv, st.d)
    err = ints([0])
    q = P.cuda(st.q)
    got = api.chunk_mass_quant(q, st.pool, table, lse, plan, dev_err=err)
    again = api.chunk_mass_quant(q, st.pool, table, lse, plan)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.equal(got, again)
    got, lse = got.cpu().to(torch.float64).numpy(), lse.cpu().to(torch.float64).numpy()
    for b in range(len(st.cu_lq) - 1):
        a, z, n0, n1 = st.cu_lq[b], st.cu_lq[b + 1], st.cu_k[b], st.cu_k[b + 1]
        if a == z:
            assert (got[n0:n1] == 0).all()
            continue
        want, tol = R.mass(f64(st.q[a:z]), pk, host, range(n0, n1), lse[a:z], 1 / math.sqrt(st.d))
        off = np.abs(got[n0:n1] - want)
        assert (off <= tol).all(), f"{off.max():.3e}, {(off / np.maximum(tol, 1e-30)).max():.2f} of its bound"


# ------------------------------------------------------------ as a program --

@pytest.mark.parametrize("fmt", FORMATS)
def test_prefill_to_reselection(fmt):
    """Prefill into a staging pool, move its slots into the 8-bit pool, select,
    decode, score every chunk and reselect; a finished block joins the cache."""
    cfg = wl.scaled(wl.CTX_8K, n_chunks=6, chunk_size=96, n_keep=40, n_select=3, n_win=8, n_resp=24)
    req = wl.make_request(cfg, 0)
    res = api.chunk_prefill(P.cuda(req["q"]), P.cuda(req["k"]), P.cuda(req["v"]),
                            P.cuda(req["q_win"]), cfg.n_chunks, cfg.chunk_size, cfg.n_keep,
                            P.cuda(req["slot_row"]), cfg.pool_rows)
    n, hq, hkv, d = cfg.n_chunks, cfg.n_q_heads, cfg.n_kv_heads, cfg.head_dim
    pool = api.QuantPool.zeros(48 * (n + 1), hkv, d, CODES[fmt])
    table = torch.zeros(n + 1, 2, dtype=torch.int32, device="cuda")
    slots = ints([48 * ((5 * j + 2) % n) for j in range(n)])
    api.pool_quantize(res["pool_k"], res["pool_v"], res["table"], pool, slots, max_len=cfg.n_keep + 1,
                      table=table[:n])
    sel, s = api.select_chunks(P.cuda(req["s_i"]), P.cuda(req["s_p"]), cfg.n_select)
    q, k, v = wl.live_block(req, wl.make_step(cfg, 0, 0))
    plan = api.QuantDecodePlan([0, cfg.n_live], [0, cfg.n_select], hq, hkv, d, cfg.n_keep + 1)
    out, lse = api.decode_attention_quant(P.cuda(q), P.cuda(k), P.cuda(v), pool, table, sel, plan)
    mass = api.chunk_mass_quant(P.cuda(q), pool, table[:n], lse,
                                api.QuantMassPlan([0, cfg.n_live], [0, n], hq, hkv, d))
    sel2, _ = api.reselect_chunks(s, mass, 10.0, ints([0, n]), ints([0, cfg.n_select]), n)
    # the live block becomes chunk n, selected alone in the next step
    api.pool_quantize(P.cuda(k), P.cuda(v), ints([[0, cfg.n_live]]), pool, ints([48 * n]),
                      max_len=cfg.n_live, table=table[n:])
    out2, lse2 = api.decode_partial_quant(
        P.cuda(q), None, None, pool, table, ints([n]),
        api.QuantDecodePlan([0, cfg.n_live], [0, 1], hq, hkv, d, cfg.n_live, self_keys=False))
    torch.cuda.synchronize()

    staged = {x: f64(res["pool_" + x].cpu()) for x in "kv"}
    src = res["table"].cpu().tolist()
    host, qv = table.cpu().numpy(), {x: values_of(pool, x) for x in "kv"}
    for x in "kv":   # what the pool holds: the staged rows, quantised
        codes, exps, written = R.quantize(staged[x], [e[1] for e in src], [e[0] for e in src],
                                          slots.cpu().tolist(), pool.rows, fmt)
        assert np.array_equal(R.values(codes, np.maximum(exps, 0))[written], qv[x][written])
    scale = 1 / math.sqrt(d)
    chunks = sel.cpu().tolist()
    want, want_lse, tol, lse_tol = R.decode(
        f64(q), np.concatenate([R.keys_of(qv["k"], host, chunks), f64(k)]),
        np.concatenate([R.keys_of(qv["v"], host, chunks), f64(v)]), scale)
    assert (np.abs(f64(out.cpu()) - want) <= tol).all()
    assert (np.abs(f64(lse.cpu()) - want_lse) <= lse_tol).all()
    m, mtol = R.mass(f64(q), qv["k"], host, range(n), f64(lse.cpu()), scale)
    assert (np.abs(f64(mass.cpu()) - m) <= mtol).all()
    ref, s2 = orc.reselect_chunks(s.cpu().numpy(), f64(mass.cpu()), 10.0, cfg.n_select)
    assert sel2.cpu().tolist() == [int(x) for x in ref]
    want, want_lse, tol, lse_tol = R.decode(f64(q), R.keys_of(qv["k"], host, [n]),
                                            R.keys_of(qv["v"], host, [n]), scale)
    assert (np.abs(f64(out2.cpu()) - want) <= tol).all()
    assert (np.abs(f64(lse2.cpu()) - want_lse) <= lse_tol).all()


@pytest.mark.parametrize("lq", [1, 16, 320])
def test_captured_and_replayed(lq):
    """A step captured into a CUDA graph, replayed on other contents."""
    st = Step("e4m3", 28, 4, 128, [lq], [[129, 65, 300]], seed=12)
    plan = api.QuantDecodePlan(st.cu_lq, st.cu_k, st.hq, st.hkv, st.d, st.max_len)
    mplan = api.QuantMassPlan(st.cu_lq, [0, st.table.shape[0]], st.hq, st.hkv, st.d)
    q, k, v = P.cuda(st.q), P.cuda(st.k_self), P.cuda(st.v_self)

    def step():
        out, lse = api.decode_attention_quant(q, k, v, st.pool, st.table, st.sel, plan)
        return out, lse, api.chunk_mass_quant(q, st.pool, st.table, lse, mplan)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (1, 2):
        g = torch.Generator().manual_seed(seed)
        q.copy_(torch.randn(q.shape, generator=g).to(torch.bfloat16))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("lq,more", [(1, 0), (40, 0), (200, 8)])
def test_two_graphs_in_turn(lq, more):
    """Two captured steps of one plan, replayed in turn and on two streams at
    once, each with workspace of its own."""
    st = Step("int8", 8, 2, 64, [lq], [[64, 40, 17] + [2049] * more], seed=18)
    plan = api.QuantDecodePlan(st.cu_lq, st.cu_k, 8, 2, 64, st.max_len, n_splits=4)
    assert plan.workspace_bytes > 0
    k, v = P.cuda(st.k_self), P.cuda(st.v_self)
    q = [P.cuda(st.q), P.cuda(-st.q)]
    want = [api.decode_attention_quant(x, k, v, st.pool, st.table, st.sel, plan) for x in q]
    torch.cuda.synchronize()
    graphs, got = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for x, graph in zip(q, graphs):
        with torch.cuda.graph(graph):
            got.append(api.decode_attention_quant(x, k, v, st.pool, st.table, st.sel, plan))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for out, lse in got:
            out.zero_(), lse.zero_()
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lqs", [(1, 4), (1, 9), (20, 40), (150, 320)])
def test_many_calls_in_a_row(lqs, fmt):
    """A ragged step again and again without a pause, three steps in turn: the
    same bits every time and no error (a wait that runs out is one)."""
    steps = []
    for seed in range(3):
        rng = np.random.RandomState(30 + seed)
        n = 24 if lqs[1] < 100 else 6
        chunks = [[int(x) for x in rng.randint(200, 514, rng.randint(3, 17))] for _ in range(n)]
        st = Step(fmt, 28, 4, 128, rng.randint(lqs[0], lqs[1] + 1, n).tolist(), chunks, seed=seed,
                  self_keys=False)
        steps.append((P.cuda(st.q), st, api.QuantDecodePlan(st.cu_lq, st.cu_k, 28, 4, 128, st.max_len,
                                                           self_keys=False)))
    err = ints([0])
    first = None
    for _ in range(60):
        got = []
        for _ in range(5):
            got += [api.decode_partial_quant(q, None, None, st.pool, st.table, st.sel, plan, dev_err=err)
                    for q, st, plan in steps]
        torch.cuda.synchronize()
        first = first or got[:3]
        assert int(err.item()) == 0
        for i, (out, lse) in enumerate(got):
            assert torch.equal(out, first[i % 3][0]) and torch.equal(lse, first[i % 3][1])


def test_given_outputs_and_workspace():
    """Outputs and a workspace that the caller keeps, one workspace for calls in
    turn; one that does not start at 256 bytes is refused."""
    st = Step("e4m3", 8, 2, 64, [40], [[64, 40, 17]], seed=19)
    plan = api.QuantDecodePlan(st.cu_lq, st.cu_k, 8, 2, 64, st.max_len, n_splits=4)
    mplan = api.QuantMassPlan(st.cu_lq, [0, st.table.shape[0]], 8, 2, 64)
    q, k, v = P.cuda(st.q), P.cuda(st.k_self), P.cuda(st.v_self)
    ws = torch.empty(max(plan.workspace_bytes, mplan.workspace_bytes) + 16, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(40, 8, device="cuda")
    mass = torch.empty(st.table.shape[0], device="cuda")
    want = api.decode_attention_quant(q, k, v, st.pool, st.table, st.sel, plan)
    want_mass = api.chunk_mass_quant(q, st.pool, st.table, want[1], mplan)
    for _ in range(3):
        api.decode_attention_quant(q, k, v, st.pool, st.table, st.sel, plan, out=out, lse=lse, workspace=ws)
        api.chunk_mass_quant(q, st.pool, st.table, lse, mplan, mass=mass, workspace=ws)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and torch.equal(mass, want_mass)
    with pytest.raises(RuntimeError):
        api.decode_attention_quant(q, k, v, st.pool, st.table, st.sel, plan, workspace=ws[16:])
    with pytest.raises(ValueError, match="workspace"):
        api.decode_attention_quant(q, k, v, st.pool, st.table, st.sel, plan, workspace=ws[:64])


def test_two_streams_at_once():
    """Calls with one plan on two streams, each with its own results."""
    st = Step("int8", 28, 4, 128, [3], [[2049] * 6], seed=13)
    want = st.run()
    plan = api.QuantDecodePlan(st.cu_lq, st.cu_k, st.hq, st.hkv, st.d, st.max_len)
    q, k, v = P.cuda(st.q), P.cuda(st.k_self), P.cuda(st.v_self)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for i in range(20):
        s = streams[i % 2]
        got.append(api.decode_attention_quant(q, k, v, st.pool, st.table, st.sel, plan,
                                              stream=s if i % 4 < 2 else s.cuda_stream))
    torch.cuda.synchronize()
    for out, lse in got:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("lq", [1, 40])
def test_temporaries_of_another_stream(lq, raw):
    """What a call is given may be dropped when it returns, although the call runs
    later, on a stream that is still busy: its memory is not handed out again before."""
    st = Step("e4m3", 8, 2, 64, [lq], [[64, 40, 17]], seed=47)
    n = st.table.shape[0]
    plan = api.QuantDecodePlan(st.cu_lq, st.cu_k, 8, 2, 64, st.max_len)
    mplan = api.QuantMassPlan(st.cu_lq, [0, n], 8, 2, 64)
    q, k, v = P.cuda(st.q), P.cuda(st.k_self), P.cuda(st.v_self)
    x, y = P.cuda(draw_rows("normal", 48, 2, 64, 1)), P.cuda(draw_rows("normal", 48, 2, 64, 2))
    want = api.decode_attention_quant(q, k, v, st.pool, st.table, st.sel, plan)
    want_mass = api.chunk_mass_quant(q, st.pool, st.table, want[1], mplan)
    pools = [api.QuantPool.zeros(48, 2, 64) for _ in range(2)]
    api.pool_quantize(x, y, ints([[0, 48]]), pools[0], ints([0]), max_len=48)
    back = api.pool_dequantize(st.pool, st.table, st.table[:, 0].contiguous(), st.pool.rows,
                               max_len=st.max_len)
    side = torch.cuda.Stream()
    at = side.cuda_stream if raw else side
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)   # about 50 ms
    got = api.decode_attention_quant(q.clone(), k.clone(), v.clone(), st.pool, st.table.clone(),
                                     st.sel.clone(), plan, stream=at)
    mass = api.chunk_mass_quant(q.clone(), st.pool, st.table.clone(), want[1].clone(), mplan, stream=at)
    api.pool_quantize(x.clone(), y.clone(), ints([[0, 48]]), pools[1], ints([0]), max_len=48, stream=at)
    rows = api.pool_dequantize(st.pool, st.table.clone(), st.table[:, 0].clone(), st.pool.rows,
                               max_len=st.max_len, stream=at)
    # takes whatever the temporaries have left
    over = [torch.full_like(t, 1) for t in (q, k, v, st.table, st.sel, want[1], x, y) for _ in range(8)]
    torch.cuda.synchronize()
    assert len(over) == 64
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(mass, want_mass)
    for a, b in zip(pools[0].tensors, pools[1].tensors):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    for row, length in st.table.cpu().tolist():   # (what no slot covers is undefined)
        for a, b in zip(rows[:2], back[:2]):
            assert torch.equal(a[row:row + length], b[row:row + length])


def test_pool_past_four_gigabytes():
    """Rows past 2^32 bytes of codes are written and read at their place."""
    hkv, d = 8, 128
    rows = (1 << 22) + 4096          # 2^32 bytes of codes and 4 MB more
    pool = api.QuantPool.zeros(rows, hkv, d)
    x, y = draw_rows("normal", 40, hkv, d, 1), draw_rows("normal", 40, hkv, d, 2)
    table = api.pool_quantize(P.cuda(x), P.cuda(y), ints([[0, 40], [0, 40]]), pool,
                              ints([rows - 48, 0]), max_len=40)
    k, v, _ = api.pool_dequantize(pool, table, ints([0, 40]), 80)
    assert torch.equal(k[:40], k[40:]) and torch.equal(v[:40], v[40:])
    codes, exps, _ = R.quantize(f64(x), [40], [0], [0], 48, "e4m3")
    assert np.array_equal(f64(k[:40].cpu()), R.values(codes, exps)[:40])
    q = P.cuda(torch.randn(3, 8, d, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16))
    for lq in (1, 3):
        plan = api.QuantDecodePlan([0, lq], [0, 1], 8, hkv, d, 40, self_keys=False)
        far = api.decode_partial_quant(q[:lq], None, None, pool, table, ints([0]), plan)
        near = api.decode_partial_quant(q[:lq], None, None, pool, table, ints([1]), plan)
        assert torch.equal(far[0], near[0]) and torch.equal(far[1], near[1])
