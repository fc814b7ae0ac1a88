"""CPU-side checks of the block-scaled E4M3 operators: the 64-bit definitions
that the GPU tests use (f8_ref.py), pinned, and what the entry points refuse
before they touch the GPU (addresses here are fake: nothing is launched)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import compressed_sparse_attention_09_b200 as csa
import f8_ref as ref

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 7
P = ctypes.c_void_p(1 << 20)         # 1024-byte aligned
ODD = ctypes.c_void_p((1 << 20) + 8)  # 8-byte aligned


# ---------------------------------------------------------------- the definitions
def test_code_table_is_torchs_e4m3():
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.TABLE, want, equal_nan=True)


def test_rounding_is_torchs_e4m3():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(20000) * 2.0 ** rng.integers(-12, 8, 20000), ref.TABLE[:127],
                        (ref.TABLE[:126] + ref.TABLE[1:127]) / 2, -(ref.TABLE[:126] + ref.TABLE[1:127]) / 2])
    x = x[np.abs(x) <= 448].astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.TABLE[ref._round_code(x.astype(np.float64))], want)


@pytest.mark.parametrize("amax,byte", [(448.0, 127), (448.0 * (1 + 2.0 ** -20), 128), (1.0, 119), (1.75, 119), (1.76, 120),
                                       (0.0, 0), (2.0 ** -149, 0), (448 * 2.0 ** -127, 0), (448 * 2.0 ** -126, 1),
                                       (3.0e38, 127 + 120)])
def test_scale_byte_by_hand(amax, byte):
    assert ref.scale_byte(amax) == byte
    if byte:
        assert amax > math.ldexp(448.0, byte - 128)


def test_quantize_by_hand():
    codes, scales = ref.quantize(np.array([[1.0, -2.0, 0.0, 3.5] + [0.0] * 12, [np.inf, np.nan, 7.0, 0.0] + [0.0] * 12]), 0)
    # row 0: A = 3.5 = 1.75 * 2: byte 120 (2^-7); 3.5 * 128 = 448
    assert scales[:, 0].tolist() == [120, 121] and ref.TABLE[codes[0, :4]].tolist() == [128.0, -256.0, 0.0, 448.0]
    assert codes[1, 0] == 0x7F and codes[1, 1] == 0x7F and ref.TABLE[codes[1, 2]] == 448.0


def test_attention_definition_on_one_and_two_entries():
    codes = torch.zeros(3, 512, dtype=torch.uint8)
    codes[0], codes[1] = 0x38, 0x40                     # 1, 2
    scales = torch.tensor([127, 126, 127], dtype=torch.uint8)
    q = torch.zeros(2, 512, dtype=torch.float64)
    o, b = ref.mqa(q, codes, scales, torch.tensor([1]), torch.bfloat16)
    assert torch.equal(o, torch.ones(2, 512, dtype=torch.float64)) and (b < 0.02).all()
    o, _ = ref.mqa(q, codes, scales, torch.tensor([0, 2]), torch.bfloat16)   # a zero entry halves the mean
    assert torch.equal(o, torch.full((2, 512), 0.5, dtype=torch.float64))
    o, b = ref.mqa(q, codes, scales, torch.tensor([], dtype=torch.long), torch.bfloat16)
    assert (o == 0).all() and (b == 0).all()


# ---------------------------------------------------------------- refusals
def launches(f):
    n0 = csa.csa_launch_count()
    rc = f()
    assert csa.csa_launch_count() == n0
    return rc


@pytest.mark.parametrize("change,status", [
    (dict(dtype=5), INVALID), (dict(X=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID),
    (dict(n=-1), INVALID), (dict(w=0), INVALID), (dict(ld=504), INVALID), (dict(ld_codes=504), INVALID),
    (dict(block=128, ld_scales=3), INVALID), (dict(ld_scales=0), INVALID), (dict(slots=P, n_slots=-1), INVALID),
    (dict(block=64), UNSUPPORTED), (dict(w=504), UNSUPPORTED), (dict(w=(1 << 28) + 16, ld=1 << 30, ld_codes=1 << 30), UNSUPPORTED), (dict(ld=516), UNSUPPORTED),
    (dict(ld_codes=520), UNSUPPORTED), (dict(X=ODD), UNSUPPORTED), (dict(codes=ODD), UNSUPPORTED), (dict(n=0), OK)])
def test_quantize_refusals(change, status):
    a = dict(dtype=csa.CSA_BF16, X=P, ld=512, n=4, w=512, block=0, slots=None, n_slots=0, codes=P, ld_codes=512, scales=P,
             ld_scales=1)
    a.update(change)
    assert launches(lambda: csa.lib().csa_quantize_f8(*a.values(), None)) == status


@pytest.mark.parametrize("change,status", [
    (dict(dtype=5), INVALID), (dict(X=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID),
    (dict(n=-1), INVALID), (dict(w=0), INVALID), (dict(ld=504), INVALID), (dict(ld_codes=504), INVALID),
    (dict(n_slots=-1), INVALID), (dict(rows=None, n=11), INVALID), (dict(block=128, ld_scales=3), INVALID),
    (dict(block=100), UNSUPPORTED), (dict(w=500), UNSUPPORTED), (dict(ld=516), UNSUPPORTED), (dict(X=ODD), UNSUPPORTED),
    (dict(codes=ODD), UNSUPPORTED), (dict(n=0), OK)])
def test_dequantize_refusals(change, status):
    a = dict(dtype=csa.CSA_BF16, codes=P, ld_codes=512, scales=P, ld_scales=1, n_slots=10, w=512, block=0, rows=P, n=4, X=P,
             ld=512)
    a.update(change)
    assert launches(lambda: csa.lib().csa_dequantize_f8(*a.values(), None)) == status


@pytest.mark.parametrize("change,status", [
    (dict(dtype=2), INVALID), (dict(W=None), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(ld=200), INVALID),
    (dict(ld_codes=200), INVALID), (dict(ld_scales=1), INVALID), (dict(K=250), UNSUPPORTED), (dict(W=ODD), UNSUPPORTED),
    (dict(ld=260), UNSUPPORTED), (dict(ld_codes=264), UNSUPPORTED)])
def test_quantize_weight_refusals(change, status):
    a = dict(dtype=csa.CSA_BF16, W=P, ld=256, N=10, K=256, codes=P, ld_codes=256, scales=P, ld_scales=2)
    a.update(change)
    assert launches(lambda: csa.lib().csa_quantize_weight_f8(*a.values(), None)) == status


@pytest.mark.parametrize("change,status", [
    (dict(out=3), INVALID), (dict(A=None), INVALID), (dict(sB=None), INVALID), (dict(D=None), INVALID), (dict(M=-1), INVALID),
    (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(lda=4080), INVALID), (dict(ldb=4080), INVALID), (dict(ldd=4159), INVALID),
    (dict(ld_sA=31), INVALID), (dict(ld_sB=31), INVALID), (dict(lda=4104), UNSUPPORTED), (dict(A=ODD), UNSUPPORTED),
    (dict(B=ODD), UNSUPPORTED), (dict(D=ctypes.c_void_p((1 << 20) + 1)), INVALID), (dict(ws=None), WORKSPACE),
    (dict(ws_bytes=1000), WORKSPACE), (dict(ws=ODD), INVALID), (dict(M=0), OK)])
def test_gemm_refusals(change, status):
    a = dict(out=csa.CSA_BF16, A=P, lda=4096, sA=P, ld_sA=32, B=P, ldb=4096, sB=P, ld_sB=32, M=64, N=4160, K=4096, D=P,
             ldd=4160, ws=P, ws_bytes=1 << 30)
    a.update(change)
    assert launches(lambda: csa.lib().csa_gemm_f8(*a.values(), None)) == status


DIMS = csa.Dims(d=256, c=512, m=4, cI=128, nhI=64, nh=128, dc=128, topk=2048, dtype=csa.CSA_BF16)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(idx=None), INVALID),
    (dict(pos=None), INVALID), (dict(O=None), INVALID), (dict(cap=0), INVALID), (dict(B=-1), INVALID),
    (dict(ld_q=65528), INVALID), (dict(ld_q=65540), UNSUPPORTED), (dict(q=ODD), UNSUPPORTED), (dict(codes=ODD), UNSUPPORTED),
    (dict(O=ODD), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(ws_bytes=100), WORKSPACE), (dict(ws=ODD), INVALID),
    (dict(B=0), OK)])
def test_decode_mqa_refusals(change, status):
    a = dict(q=P, ld_q=65536, codes=P, scales=P, idx=P, pos=P, cap=100, B=1, O=P, ws=P, ws_bytes=1 << 30)
    a.update(change)
    d = ctypes.byref(DIMS.c_struct())
    assert launches(lambda: csa.lib().csa_decode_mqa_f8(d, *a.values(), None)) == status


@pytest.mark.parametrize("change,status", [
    (dict(cu=None), INVALID), (dict(cb=None), INVALID), (dict(nseq=0), INVALID), (dict(T=-1), INVALID), (dict(NB=-1), INVALID),
    (dict(q=ODD), UNSUPPORTED), (dict(T=0), OK)])
def test_sparse_mqa_refusals(change, status):
    a = dict(q=P, ld_q=65536, codes=P, scales=P, idx=P, cu=P, cb=P, nseq=1, T=500, NB=125, O=P, ws=None, ws_bytes=0)
    a.update(change)
    d = ctypes.byref(DIMS.c_struct())
    assert launches(lambda: csa.lib().csa_sparse_mqa_f8(d, *a.values(), None)) == status


def test_decode_step_and_append_refusals():
    L, d = csa.lib(), ctypes.byref(DIMS.c_struct())
    need = csa.csa_decode_f8_workspace_bytes(DIMS, 2, 100)
    assert need > csa.csa_decode_workspace_bytes(DIMS, 2, 100)
    step = lambda ws=P, n=need, h=P, dims=d: L.csa_decode_f8(dims, P, P, h, P, P, P, P, P, P, P, 100, 2, P, None, ws, n, None)  # noqa: E731
    assert launches(lambda: step(n=need - 1)) == WORKSPACE
    assert launches(lambda: step(ws=None)) == INVALID
    assert launches(lambda: step(ws=ODD)) == INVALID
    assert launches(lambda: step(h=ODD)) == UNSUPPORTED
    for change in (dict(dtype=csa.CSA_F32), dict(cI=64), dict(nhI=16), dict(d=264)):
        bad = csa.Dims(**{**{f: getattr(DIMS, f) for f in ("d", "c", "m", "cI", "nhI", "nh", "dc", "topk", "dtype")}, **change})
        assert csa.csa_decode_f8_workspace_bytes(bad, 2, 100) == 0
        assert launches(lambda: step(dims=ctypes.byref(bad.c_struct()), n=1 << 30)) == UNSUPPORTED
    assert launches(lambda: L.csa_cache_append_f8(d, P, P, P, P, None, P, P, P, P, 100, 2, None)) == INVALID
    assert launches(lambda: L.csa_cache_append_f8(d, P, P, P, P, ODD, P, P, P, P, 100, 2, None)) == UNSUPPORTED
    assert launches(lambda: L.csa_cache_append_f8(d, P, P, P, P, P, P, P, P, P, 100, 0, None)) == OK


def test_packed_weights_sizes_and_refusals():
    L, d = csa.lib(), ctypes.byref(DIMS.c_struct())
    n1, n2 = 4 * 512 + 4 * 128 + 128 + 64, 64 * 128 + 128 * 512
    need = csa.csa_packed_weights_f8_bytes(DIMS)
    assert need >= n1 * 256 + n2 * 128
    assert launches(lambda: L.csa_pack_weights_f8(d, P, P, need - 1, None)) == WORKSPACE
    assert launches(lambda: L.csa_pack_weights_f8(d, P, None, need, None)) == INVALID
    assert launches(lambda: L.csa_pack_weights_f8(d, P, ODD, need, None)) == INVALID
    f32 = csa.Dims(d=256, c=64, m=4, cI=32, nhI=4, nh=8, dc=128, topk=16, dtype=csa.CSA_F32)
    assert csa.csa_packed_weights_f8_bytes(f32) == 0
    assert launches(lambda: L.csa_pack_weights_f8(ctypes.byref(f32.c_struct()), P, P, need, None)) == UNSUPPORTED


def test_workspace_sizes():
    """Few rows are split (K slices of the product, entries of the attention): only then a workspace is needed."""
    assert csa.csa_gemm_f8_workspace_bytes(64, 4160, 4096) >= 2 * 4160 * 64 * 4
    assert csa.csa_gemm_f8_workspace_bytes(8192, 4160, 4096) == 0
    assert csa.csa_gemm_f8_workspace_bytes(0, 4160, 4096) == 0
    assert csa.csa_mqa_f8_workspace_bytes(DIMS, 1) >= 2 * 128 * 512 * 4
    assert csa.csa_mqa_f8_workspace_bytes(DIMS, 8192) == 0
    simt = csa.Dims(d=64, c=64, m=4, cI=32, nhI=4, nh=8, dc=64, topk=16, dtype=csa.CSA_F32)
    assert csa.csa_mqa_f8_workspace_bytes(simt, 1) == 0
