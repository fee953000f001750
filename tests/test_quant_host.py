"""CPU tests of the 8-bit chunk pool: its calls refuse bad arguments on the
host before anything is launched, the Python layer refuses tensors of the
wrong place, type or shape before it reaches the library, and the reference
of the GPU tests is checked against torch's own conversions."""
import ctypes
import os

import numpy as np
import pytest
import torch

import __graft_entry__ as entry
from sparse_chunked_kv_gb300 import _abi, api, quant
from tests import quant_reference as R

INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_abi.LIB_PATH):
        entry.build()
    return _abi.load()


def _call(lib, name, args, over):
    assert set(over) <= set(args), over
    a = dict(args, **over)
    return getattr(lib, name)(*[x if x != 0 or not k.startswith("p_") else None
                                for k, x in a.items()])


QUANTIZE = dict(p_k=256, p_v=256, src_rows=40, p_src=256, n=2, max_len=16, Hkv=2, D=64, fmt=0,
                p_pk=256, p_pv=256, p_ek=256, p_ev=256, rows=64, p_slot=256, p_table=512, p_err=0,
                stream=None)
DEQUANTIZE = dict(p_pk=256, p_pv=256, p_ek=256, p_ev=256, rows=64, p_table=256, table_len=2, p_sel=0,
                  n=2, max_len=16, Hkv=2, D=64, fmt=0, p_k=256, p_v=256, dst_rows=40, p_dst=256,
                  p_dt=0, p_err=0, stream=None)

COMMON = [(dict(p_k=0), INVALID), (dict(p_v=0), INVALID), (dict(p_pk=0), INVALID),
          (dict(p_ev=0), INVALID), (dict(p_ek=0), INVALID), (dict(p_table=0), INVALID),
          (dict(n=0), INVALID), (dict(max_len=0), INVALID), (dict(Hkv=0), INVALID),
          (dict(D=96), UNSUPPORTED), (dict(fmt=2), INVALID), (dict(fmt=-1), INVALID),
          (dict(rows=40), INVALID), (dict(rows=0), INVALID), (dict(rows=1 << 31), UNSUPPORTED),
          (dict(p_k=264), INVALID), (dict(p_pv=264), INVALID),
          (dict(n=1 << 30, max_len=40, Hkv=4096), UNSUPPORTED)]


@pytest.mark.parametrize("over,status", COMMON + [
    (dict(p_src=0), INVALID), (dict(p_slot=0), INVALID), (dict(src_rows=0), INVALID),
    (dict(src_rows=1 << 31), UNSUPPORTED)])
def test_quantize_host_checks(lib, over, status):
    assert _call(lib, "pfd_pool_quantize", QUANTIZE, over) == status


@pytest.mark.parametrize("over,status", [(o, s) for o, s in COMMON if "n" not in o or o["n"] == 0] + [
    (dict(p_dst=0), INVALID), (dict(dst_rows=0), INVALID), (dict(table_len=0), INVALID),
    (dict(table_len=1), INVALID),
    (dict(n=1 << 30, max_len=40, Hkv=4096, p_sel=256), UNSUPPORTED)])
def test_dequantize_host_checks(lib, over, status):
    assert _call(lib, "pfd_pool_dequantize", DEQUANTIZE, over) == status


@pytest.mark.parametrize("name,args,written,read", [
    ("pfd_pool_quantize", QUANTIZE, "p_table", ("p_src", "p_slot")),
    ("pfd_pool_dequantize", DEQUANTIZE, "p_dt", ("p_table", "p_sel", "p_dst"))])
def test_the_written_table_is_apart_from_what_is_read(lib, name, args, written, read):
    """Two entries of 8 bytes that begin before, at and inside the other's."""
    for other in read:
        for at in (1008, 1016, 1020):
            over = {written: 1016, other: at}
            if at == 1008 and other not in ("p_src", "p_table"):
                over[other] = 1012            # (two of 4 bytes)
            assert _call(lib, name, args, over) == INVALID, (other, at)


def test_no_entries_share_nothing():
    t = _i32(8, 2)
    quant._apart(t[3:3], "dst_table", table=t)
    quant._apart(t[3:5], "dst_table", table=t[4:4], sel=t[:3].view(-1), dst_row=None)


def test_shared_entries_are_refused(monkeypatch):
    monkeypatch.setattr(quant, "_need", lambda *a: None)
    _no_library(monkeypatch)
    t = _i32(8, 2)
    with pytest.raises(ValueError, match="src_table"):
        api.pool_quantize(_bf(8, 2, 64), _bf(8, 2, 64), t[:3], _Pool, _i32(3), max_len=8, table=t[2:5])
    with pytest.raises(ValueError, match="slot_row"):
        api.pool_quantize(_bf(8, 2, 64), _bf(8, 2, 64), t[:3], _Pool, t[4:6].view(-1)[:3], max_len=8,
                          table=t[3:6])
    for name, kw in (("table", dict(dst_table=t[7:8])), ("sel", dict(dst_table=_i32(1, 2)))):
        if name == "sel":
            kw["sel"] = kw["dst_table"].view(-1)[1:]
        with pytest.raises(ValueError, match=name):
            api.pool_dequantize(_Pool, t, _i32(1), 8, max_len=8, **dict(dict(sel=_i32(1)), **kw))


def _host(*values):
    return ctypes.cast((ctypes.c_int32 * len(values))(*values), ctypes.c_void_p)


LQ, KS = _host(0, 4, 8), _host(0, 1, 3)
DECODE = dict(p_q=256, p_ks=256, p_vs=256, p_lq=256, lq=LQ, fmt=0, p_pk=256, p_pv=256, p_ek=256,
              p_ev=256, rows=64, p_table=256, table_len=4, p_sel=256, p_cuk=256, ks=KS, batch=2, Hq=4,
              Hkv=2, D=64, longest=20, scale=0.0, splits=0, p_out=256, p_lse=256, p_err=0, p_ws=256,
              bytes=1 << 24, stream=None)
DECODE_BAD = [
    (dict(p_q=0), INVALID), (dict(p_lq=0), INVALID), (dict(p_pk=0), INVALID), (dict(p_pv=0), INVALID),
    (dict(p_ek=0), INVALID), (dict(p_ev=0), INVALID), (dict(p_table=0), INVALID),
    (dict(p_sel=0), INVALID), (dict(p_cuk=0), INVALID), (dict(p_out=0), INVALID),
    (dict(fmt=2), INVALID), (dict(fmt=-1), INVALID), (dict(rows=40), INVALID), (dict(rows=0), INVALID),
    (dict(rows=1 << 31), UNSUPPORTED), (dict(table_len=0), INVALID), (dict(batch=0), INVALID),
    (dict(Hq=5), INVALID), (dict(D=96), UNSUPPORTED), (dict(Hq=258, Hkv=2), UNSUPPORTED),
    (dict(longest=-1), INVALID), (dict(splits=65), INVALID), (dict(splits=-1), INVALID), (dict(splits=8, bytes=64), INVALID),
    (dict(splits=8, p_ws=0, bytes=0), INVALID), (dict(p_ws=300), INVALID), (dict(p_q=264), INVALID),
    (dict(p_pk=264), INVALID), (dict(p_out=264), INVALID), (dict(lq=None), INVALID),
    (dict(lq=_host(0, 4, 3)), INVALID), (dict(ks=_host(0, 1, 0)), INVALID),
    (dict(ks=_host(0, 600, 600)), UNSUPPORTED), (dict(lq=_host(0, 0, 0)), INVALID)]


@pytest.mark.parametrize("over,status", DECODE_BAD + [(dict(p_ks=0), INVALID), (dict(p_vs=0), INVALID)])
def test_decode_host_checks(lib, over, status):
    assert _call(lib, "pfd_decode_attention_quant", DECODE, over) == status


@pytest.mark.parametrize("over,status", DECODE_BAD + [
    (dict(p_lse=0), INVALID), (dict(self_keys=2), INVALID), (dict(p_ks=0, self_keys=1), INVALID)])
def test_decode_partial_host_checks(lib, over, status):
    args = {}
    for k, x in DECODE.items():
        if k == "splits":
            args["self_keys"] = 0
        args[k] = x
    assert _call(lib, "pfd_decode_partial_quant", args, over) == status


STAGED = dict(lq=_host(0, 400, 800), ks=_host(0, 8, 16), Hq=28, Hkv=4, D=128, longest=2049,
              rows=4096, bytes=1 << 40)


@pytest.mark.parametrize("lq", [1, 40])
def test_more_key_groups_than_the_kernels_count(lib, lq):
    """One chunk may be selected many times: 17 or more of 2^31 - 16 rows are over
    2^31 groups of 16, and a bound past the pool's rows counts as these."""
    args = dict(DECODE, lq=_host(0, lq, lq), rows=(1 << 31) - 16, longest=2 ** 31 - 1, bytes=1 << 40)
    assert _call(lib, "pfd_decode_attention_quant", args, dict(ks=_host(0, 17, 17))) == UNSUPPORTED
    for over in (dict(ks=_host(0, 15, 30)), dict(ks=_host(0, 17, 17), rows=64)):
        # (a workspace that does not start at 256 bytes ends the call at the next check)
        assert _call(lib, "pfd_decode_attention_quant", args, dict(over, p_ws=300)) == INVALID


@pytest.mark.parametrize("splits", [1, 2])
@pytest.mark.parametrize("partial", [False, True])
def test_a_staged_step_needs_its_workspace(lib, partial, splits):
    """Many rows: the chunks are read back to the workspace, with one split too,
    where no partial outputs need one."""
    args = dict(DECODE, **STAGED, splits=splits)
    need = _abi.pfd_decode_quant_workspace(2, [0, 400, 800], [0, 8, 16], 28, 4, 128, 2049, 1, splits)
    assert need >= 16 * 2049 * 4 * 4 * 128
    if partial:
        items = list(args.items())
        at = [k for k, _ in items].index("splits")
        args = dict(items[:at] + [("self_keys", 1)] + items[at:])
    name = "pfd_decode_partial_quant" if partial else "pfd_decode_attention_quant"
    for over in (dict(p_ws=0), dict(bytes=need - 1), dict(p_ws=128)):
        assert _call(lib, name, args, over) == INVALID, over


@pytest.mark.parametrize("over,status", [
    (dict(p_q=0), INVALID), (dict(p_pk=0), INVALID), (dict(p_ek=0), INVALID), (dict(p_lse=0), INVALID),
    (dict(p_mass=0), INVALID), (dict(fmt=2), INVALID), (dict(rows=40), INVALID),
    (dict(rows=1 << 31), UNSUPPORTED), (dict(D=96), UNSUPPORTED), (dict(Hq=5), INVALID),
    (dict(table_len=2), INVALID), (dict(bytes=16), INVALID), (dict(p_ws=0), INVALID),
    (dict(p_pk=264), INVALID), (dict(batch=65), UNSUPPORTED), (dict(ns=_host(0, 2, 1)), INVALID)])
def test_mass_host_checks(lib, over, status):
    args = dict(p_q=256, p_lq=256, lq=LQ, fmt=1, p_pk=256, p_ek=256, rows=64, p_table=256, table_len=4,
                ns=KS, p_lse=256, batch=2, Hq=4, Hkv=2, D=64, scale=0.0, p_mass=256, p_err=0, p_ws=256,
                bytes=1 << 20, stream=None)
    assert _call(lib, "pfd_chunk_mass_quant", args, over) == status


def test_workspace_holds_fp32_partials():
    """Two splits: max and denominator and D fp32 outputs per (row, head)."""
    one = _abi.pfd_decode_quant_workspace(2, [0, 4, 8], [0, 1, 3], 4, 2, 64, 20, 1, 1)
    two = _abi.pfd_decode_quant_workspace(2, [0, 4, 8], [0, 1, 3], 4, 2, 64, 20, 1, 2)
    assert one == 0 and two == 2 * (2 * 8 * 4 * 4) + 2 * 8 * 4 * 64 * 4


def test_workspace_of_a_loose_bound():
    """A copy of the selected chunks is planned for many rows, and not where the
    bound of their lengths makes it larger than 8e9 bytes."""
    def need(longest):
        return _abi.pfd_decode_quant_workspace(2, [0, 300, 600], [0, 8, 16], 28, 4, 128, longest, 1, 1)
    copy = 16 * 4096 * 4 * 128 * 2 * 2
    assert copy <= need(4096) <= copy + 1024
    assert need(1 << 20) == 0 and need(2 ** 31 - 1) == 0


@pytest.mark.parametrize("hq,hkv,d,batch,chunks,rows,lq,staged", [
    (28, 4, 128, 16, 16, 257, 108, False), (28, 4, 128, 16, 16, 257, 144, True),
    (28, 4, 64, 16, 16, 257, 54, False), (28, 4, 64, 16, 16, 257, 144, True),
    (8, 2, 64, 1, 64, 257, 256, False), (8, 2, 64, 1, 64, 257, 576, True),
    (16, 16, 64, 1, 64, 257, 384, False), (16, 16, 64, 16, 16, 257, 384, True),
    (32, 8, 128, 1, 4, 257, 384, False), (32, 8, 128, 1, 4, 257, 896, True),
    (28, 4, 128, 1, 4, 257, 320, False), (28, 4, 128, 8, 8, 257, 320, True)])
def test_when_chunks_are_read_back_first(hq, hkv, d, batch, chunks, rows, lq, staged):
    """The faster of the two measured ways (the comment at stage_pays has the times),
    by the workspace that a step of one split needs: the copy of its chunks, or none."""
    need = _abi.pfd_decode_quant_workspace(batch, [lq * b for b in range(batch + 1)],
                                           [chunks * b for b in range(batch + 1)], hq, hkv, d, rows, 1, 1)
    copy = batch * chunks * rows * hkv * d * 4
    assert copy <= need < copy + (1 << 16) if staged else need == 0


@pytest.mark.parametrize("hq,hkv,d,batch,chunks,rows,few", [
    (8, 2, 128, 1, 8, 257, False), (8, 2, 128, 1, 100, 513, False), (8, 2, 128, 2, 64, 513, True),
    (8, 2, 128, 1, 64, 2049, True), (8, 2, 64, 1, 8, 257, False), (8, 2, 64, 1, 100, 513, True),
    (32, 8, 128, 1, 8, 257, False), (32, 8, 128, 4, 64, 513, True), (32, 8, 64, 4, 64, 513, True)])
def test_which_kernel_takes_17_to_32_rows(hq, hkv, d, batch, chunks, rows, few):
    """The faster of the two measured (the comment at few_rows_pays has the times).
    Each has a plan of its own for the splits: 32 rows are split as 16 are where the
    few-rows kernel takes them, else as 36 are."""
    def splits(lq):
        need = _abi.pfd_decode_quant_workspace(batch, [lq * b for b in range(batch + 1)],
                                               [chunks * b for b in range(batch + 1)], hq, hkv, d,
                                               rows, 1, 0)
        return need // (batch * lq * hq * (8 + 4 * d))
    assert hq // hkv == 4
    one, two = splits(4), splits(9)
    assert one != two
    assert splits(8) == (one if few else two)


# --------------------------------------------------------------- Python --

def _no_library(monkeypatch):
    def reached():
        raise AssertionError("the library was reached")
    monkeypatch.setattr(_abi, "load", reached)


class _Pool:
    """A pool's outline on the host (QuantPool itself takes CUDA tensors only)."""
    device, n_kv_heads, head_dim, rows, format = torch.device("cuda", 0), 2, 64, 32, 0
    k = v = exp_k = exp_v = None
    tensors = ()


class _Plan:
    device, n_kv_heads, n_q_heads, head_dim = torch.device("cuda", 0), 2, 4, 64
    total_lq, total_chunks, self_keys, complete = 3, 1, True, True
    tensors = ()


def _bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def _i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


CALLS = {
    "pool_quantize": lambda: api.pool_quantize(_bf(8, 2, 64), _bf(8, 2, 64), _i32(1, 2), _Pool,
                                               _i32(1), max_len=8),
    "pool_dequantize": lambda: api.pool_dequantize(_Pool, _i32(1, 2), _i32(1), 8, max_len=8),
    "decode_attention_quant": lambda: api.decode_attention_quant(
        _bf(3, 4, 64), _bf(3, 2, 64), _bf(3, 2, 64), _Pool, _i32(1, 2), _i32(1), _Plan),
    "decode_partial_quant": lambda: api.decode_partial_quant(
        _bf(3, 4, 64), None, None, _Pool, _i32(1, 2), _i32(1), _Plan),
    "chunk_mass_quant": lambda: api.chunk_mass_quant(_bf(3, 4, 64), _Pool, _i32(1, 2),
                                                     torch.zeros(3, 4), _Plan),
    "QuantPool": lambda: api.QuantPool(torch.zeros(32, 2, 64, dtype=torch.int8),
                                       torch.zeros(32, 2, 64, dtype=torch.int8),
                                       torch.zeros(2, 2, dtype=torch.uint8),
                                       torch.zeros(2, 2, dtype=torch.uint8)),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_calls_refuse_host_tensors(name, monkeypatch):
    _no_library(monkeypatch)
    with pytest.raises(ValueError, match="CUDA"):
        CALLS[name]()


def test_codes_of_another_type_are_refused():
    with pytest.raises(ValueError, match="codes"):
        api.QuantPool(_bf(32, 2, 64), _bf(32, 2, 64), _i32(2, 2), _i32(2, 2))


def test_a_pool_keeps_its_tensors(monkeypatch):
    """Others cannot take their places unchecked, and no address outlives its memory."""
    monkeypatch.setattr(quant, "_need", lambda *a: None)
    codes = type("Codes", (), dict(dtype=torch.int8, is_cuda=True, device=torch.device("cuda", 0),
                                   shape=(32, 2, 64), at=1, dim=lambda s: 3,
                                   data_ptr=lambda s: s.at))
    parts = [codes() for _ in range(4)]
    pool = api.QuantPool(*parts)
    assert (pool.k, pool.v, pool.exp_k, pool.exp_v) == tuple(parts)
    for name in ("k", "v", "exp_k", "exp_v"):
        with pytest.raises(AttributeError):
            setattr(pool, name, codes())
    assert pool.pointers == (1, 1, 1, 1)
    parts[2].at = 5
    assert pool.pointers == (1, 1, 5, 1)


@pytest.mark.parametrize("cu_lq,cu_k", [([0, 2, 1], [0, 1, 2]), ([0, 2], [0, 1, 2]), ([1, 2], [0, 1]),
                                        ([0], [0])])
def test_plans_refuse_malformed_counts(cu_lq, cu_k):
    with pytest.raises(ValueError):
        api.QuantDecodePlan(cu_lq, cu_k, 4, 2, 64, 20)
    with pytest.raises(ValueError):
        api.QuantMassPlan(cu_lq, cu_k, 4, 2, 64)


def test_a_partial_plan_is_not_a_whole_step():
    plan = type("P", (_Plan,), dict(self_keys=False))
    with pytest.raises(ValueError, match="partial"):
        api.decode_attention_quant(None, None, None, _Pool, None, None, plan)


@pytest.mark.parametrize("rows", [dict(dst_rows=0), dict(dst_rows=-1),
                                  dict(k=_bf(0, 2, 64), v=_bf(0, 2, 64))])
def test_reading_slots_back_needs_rows(rows, monkeypatch):
    """Without a destination row nothing would say where the slots are."""
    _no_library(monkeypatch)
    with pytest.raises(ValueError, match="dst_rows"):
        api.pool_dequantize(_Pool, _i32(1, 2), _i32(1), max_len=8, **rows)


def test_a_stream_of_another_device_is_refused(monkeypatch):
    """Its device would become the current one, with every pointer on the pool's."""
    monkeypatch.setattr(quant, "_need", lambda *a: None)
    _no_library(monkeypatch)
    other = type("Stream", (), dict(device=torch.device("cuda", 1)))()
    for call in (
            lambda: api.pool_quantize(_bf(8, 2, 64), _bf(8, 2, 64), _i32(1, 2), _Pool, _i32(1),
                                      max_len=8, stream=other),
            lambda: api.pool_dequantize(_Pool, _i32(1, 2), _i32(1), 8, max_len=8, stream=other),
            lambda: api.decode_partial_quant(_bf(3, 4, 64), None, None, _Pool, _i32(1, 2), _i32(1),
                                             type("P", (_Plan,), dict(self_keys=False, given_workspace=lambda s, w: w))(),
                                             stream=other)):
        with pytest.raises(ValueError, match="stream"):
            call()


def test_api_offers_the_module():
    for name in ("QuantPool", "QuantDecodePlan", "QuantMassPlan", "pool_quantize", "pool_dequantize",
                 "decode_attention_quant", "decode_partial_quant", "chunk_mass_quant"):
        assert getattr(api, name) is getattr(quant, name)


# ------------------------------------------------------------- reference --

def test_reference_rounds_as_torch_does():
    """E4M3 codes of every bf16 up to 448 and integer codes up to 127 equal
    torch's conversions; every code keeps its value."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16)
    x = bits.view(torch.bfloat16).float()
    x = x[torch.isfinite(x) & (x.abs() <= 448)]
    want = x.to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.round_code(x.double().numpy(), "e4m3"), want)
    x = x[x.abs() <= 127]
    assert np.array_equal(R.round_code(x.double().numpy(), "int8"), x.round().double().numpy())
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    codes = codes[torch.isfinite(codes)].numpy()
    assert np.array_equal(R.round_code(codes, "e4m3"), codes)


@pytest.mark.parametrize("fmt,top,e", [("e4m3", 448.0, 0), ("e4m3", 450.0, 1), ("e4m3", 0.0, -100),
                                       ("int8", 127.0, 0), ("int8", 127.5, 1), ("int8", 3.96875, -5),
                                       ("int8", 4.0, -4), ("e4m3", 2.0 ** -120, -100)])
def test_reference_scale(fmt, top, e):
    assert R.scale_exponents(np.full((1, 1, 1), top), fmt)[0] == e
