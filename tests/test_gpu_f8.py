"""The block-scaled E4M3 operators (csa_quantize_f8, csa_dequantize_f8,
csa_quantize_weight_f8, csa_gemm_f8, csa_sparse_mqa_f8, csa_decode_mqa_f8)
against their definitions in 64 bits (f8_ref.py): conversions bit for bit,
products and attention within bounds derived there."""
import numpy as np
import pytest
import torch

import compressed_sparse_attention_09_b200 as csa
import f8_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
KIND = {BF16: csa.CSA_BF16, F32: csa.CSA_F32}


def rows_of(rng, n, w, dtype):
    """Rows of unequal magnitude with zeros, powers of two at the scale's border, tiny and non-finite values."""
    x = rng.standard_normal((n, w)) * np.exp2(rng.integers(-30, 30, (n, 1)))
    x[rng.random((n, w)) < 0.05] = 0
    if n > 3:
        x[0] = 0
        x[1, :] = 0
        x[1, w // 2] = 448 * 2.0 ** -3              # exactly the largest code
        x[2, 0] = 448 * 2.0 ** 5 * (1 + 2.0 ** -7)   # just above: the next scale
        x[3] = np.exp2(rng.integers(-40, 3, w).astype(float))
    return torch.as_tensor(x, dtype=torch.float32).to(dtype)


# ---------------------------------------------------------------- rows
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,w,block", [(1, 16, 0), (5, 512, 0), (67, 512, 128), (33, 1040, 0), (19, 1056, 128),
                                       (1, 128, 128), (4, 144, 128), (1000, 64, 0), (7, 4096, 128), (3, 2064, 0)])
def test_quantize_bit_for_bit(n, w, block, dtype):
    rng = np.random.default_rng(n + w)
    x = rows_of(rng, n, w, dtype)
    if n > 4:
        x[4, 1], x[4, w - 1] = float("inf"), float("nan")
        if n > 5:
            x[5, w // 2] = float("nan")
        if n > 6:
            x[6, :] = float("-inf")
    nb = -(-w // block) if block else 1
    src = torch.zeros(n, w + 16, dtype=dtype, device=DEV)      # strided source and destinations
    src[:, :w] = x.to(DEV)
    codes = torch.full((n, w + 32), 0xA5, dtype=torch.uint8, device=DEV)
    scales = torch.full((n, nb + 3), 0xA5, dtype=torch.uint8, device=DEV)
    csa.csa_quantize_f8(KIND[dtype], src, w + 16, n, w, block, None, 0, codes, w + 32, scales, nb + 3)
    assert csa.csa_get_device_status() == 0
    want, ws = ref.quantize(x.double().numpy(), block)
    assert np.array_equal(codes[:, :w].cpu().numpy(), want)
    assert np.array_equal(scales[:, :nb].cpu().numpy(), ws)
    assert (codes[:, w:] == 0xA5).all() and (scales[:, nb:] == 0xA5).all()


@pytest.mark.parametrize("block", [0, 128])
def test_quantize_into_slots(block):
    """Rows land where `slots` says, -1 rows nowhere, unnamed rows keep their bytes, a bad slot is flagged."""
    rng = np.random.default_rng(3)
    n, w, rows = 50, 256, 90
    x = rows_of(rng, n, w, BF16)
    slots = torch.as_tensor(rng.permutation(rows)[:n].astype(np.int32))
    slots[7] = -1
    nb = 2 if block else 1
    codes = torch.full((rows, w), 0xA5, dtype=torch.uint8, device=DEV)
    scales = torch.full((rows, nb), 0xA5, dtype=torch.uint8, device=DEV)
    csa.csa_quantize_f8(csa.CSA_BF16, x.to(DEV), w, n, w, block, slots.to(DEV), rows, codes, w, scales, nb)
    assert csa.csa_get_device_status() == 0
    want, ws = np.full((rows, w), 0xA5, np.uint8), np.full((rows, nb), 0xA5, np.uint8)
    c, s = ref.quantize(x.double().numpy(), block)
    for i, k in enumerate(slots.tolist()):
        if k >= 0:
            want[k], ws[k] = c[i], s[i]
    assert np.array_equal(codes.cpu().numpy(), want) and np.array_equal(scales.cpu().numpy(), ws)
    for bad in (rows, -2, 2 ** 31 - 1):
        slots[7] = bad
        csa.csa_quantize_f8(csa.CSA_BF16, x.to(DEV), w, n, w, block, slots.to(DEV), rows, codes, w, scales, nb)
        assert csa.csa_get_device_status() == 5   # CSA_ERR_BAD_INDEX
        assert np.array_equal(codes.cpu().numpy(), want)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,w,block", [(1, 16, 0), (300, 512, 0), (33, 1040, 128), (7, 4096, 128), (100, 48, 0)])
def test_read_back_exact(n, w, block, dtype):
    rng = np.random.default_rng(n)
    rows, nb = 77, -(-w // block) if block else 1
    codes = torch.as_tensor(rng.integers(0, 256, (rows, w)).astype(np.uint8))
    scales = torch.as_tensor(rng.integers(90, 150, (rows, nb)).astype(np.uint8))
    scales[0] = 0                                     # 2^-127: subnormal
    at = torch.as_tensor(rng.integers(0, rows, n).astype(np.int32))
    at[0] = 0
    if n > 2:
        at[1], at[2] = -1, rows - 1
    out = torch.full((n, w + 8), 7.0, dtype=dtype, device=DEV)
    csa.csa_dequantize_f8(KIND[dtype], codes.to(DEV), w, scales.to(DEV), nb, rows, w, block, at.to(DEV), n, out, w + 8)
    assert csa.csa_get_device_status() == 0
    want = ref.decode(codes, scales, block)[at.clamp(min=0).long()]
    want[at < 0] = 0
    got = out[:, :w].cpu().double()
    if dtype == F32:
        assert torch.equal(torch.nan_to_num(got, nan=1e9), torch.nan_to_num(want, nan=1e9))
    else:   # exact but for subnormal bf16
        assert torch.equal(torch.nan_to_num(got, nan=1e9), torch.nan_to_num(want.to(F32).to(BF16).double(), nan=1e9))
        big = want.abs() > 2.0 ** -120
        assert torch.equal(got[big], want[big])
    assert (out[:, w:] == 7).all()
    at[0] = rows
    csa.csa_dequantize_f8(KIND[dtype], codes.to(DEV), w, scales.to(DEV), nb, rows, w, block, at.to(DEV), n, out, w + 8)
    assert csa.csa_get_device_status() == 5 and (out[0, :w] == 0).all()


def test_write_then_read_is_within_half_a_step():
    """A row comes back within half an E4M3 step of each value (2^-4 relative, 2^-10 of the scale below 2^-6)."""
    rng = np.random.default_rng(8)
    n, w = 64, 512
    x = torch.as_tensor(rng.standard_normal((n, w)), dtype=BF16)
    codes = torch.zeros(n, w, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(n, 1, dtype=torch.uint8, device=DEV)
    csa.csa_quantize_f8(csa.CSA_BF16, x.to(DEV), w, n, w, 0, None, 0, codes, w, scales, 1)
    out = torch.empty(n, w, dtype=BF16, device=DEV)
    csa.csa_dequantize_f8(csa.CSA_BF16, codes, w, scales, 1, n, w, 0, None, n, out, w)
    d = (out.cpu().double() - x.double()).abs()
    unit = torch.exp2(scales.cpu().double() - 127)
    assert (d <= torch.maximum(2.0 ** -4 * x.double().abs(), 2.0 ** -10 * unit)).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,K", [(1, 16), (128, 128), (130, 272), (300, 1040)])
def test_quantize_weight_bit_for_bit(N, K, dtype):
    rng = np.random.default_rng(N)
    x = torch.as_tensor(rng.standard_normal((N, K)) * np.exp2(rng.integers(-9, 9, (N, 1))), dtype=F32).to(dtype)
    kb, nb = -(-K // 128), -(-N // 128)
    codes = torch.full((N, K + 16), 0xA5, dtype=torch.uint8, device=DEV)
    scales = torch.full((nb, kb + 1), 0xA5, dtype=torch.uint8, device=DEV)
    csa.csa_quantize_weight_f8(KIND[dtype], x.to(DEV), K, N, K, codes, K + 16, scales, kb + 1)
    want, ws = ref.quantize_squares(x.double().numpy())
    assert np.array_equal(codes[:, :K].cpu().numpy(), want)
    assert np.array_equal(scales[:, :kb].cpu().numpy(), ws)
    assert (codes[:, K:] == 0xA5).all() and (scales[:, kb:] == 0xA5).all()


# ---------------------------------------------------------------- product
def gemm_case(M, N, K, dtype, seed, spread=6, pad=0, shift=0):
    g = torch.Generator().manual_seed(seed)
    lda, ldd = -(-K // 16) * 16 + 16 * pad, N + pad
    kb, nb = -(-K // 128), -(-N // 128)
    a = torch.randint(0, 256, (M, lda), generator=g).to(torch.uint8)
    b = torch.randint(0, 256, (N, lda), generator=g).to(torch.uint8)
    a[(a & 127) == 127] = 3                         # no NaN codes
    b[(b & 127) == 127] = 5
    sa = torch.randint(127 - spread, 128 + spread, (M, kb + pad), generator=g).to(torch.uint8)
    sb = torch.randint(127 - spread, 128 + spread, (nb, kb + pad), generator=g).to(torch.uint8)
    whole = torch.full((M * ldd + shift,), 5.0, dtype=dtype, device=DEV)   # the output begins `shift` values in
    out = whole[shift:].view(M, ldd)
    ws = torch.empty(csa.csa_gemm_f8_workspace_bytes(M, N, K), dtype=torch.uint8, device=DEV)
    a, b, sa, sb = (t.to(DEV) for t in (a, b, sa, sb))
    csa.csa_gemm_f8(KIND[dtype], a, lda, sa, kb + pad, b, lda, sb, kb + pad, M, N, K, out, ldd, ws)
    assert csa.csa_get_device_status() == 0
    want, bound = ref.gemm(ref.decode(a[:, :K], sa[:, :kb], 128), ref.decode_squares(b[:, :K], sb[:, :kb]), dtype)
    err = (out[:, :N].double() - want).abs()
    held = torch.isfinite(bound)
    assert held.float().mean() > 0.5
    assert (err[held] <= bound[held]).all(), (float((err / bound)[held].max()), M, N, K)
    assert (out[:, N:] == 5).all() and (whole[:shift] == 5).all()


@pytest.mark.parametrize("M,N,K", [(1, 128, 128), (3, 200, 512), (64, 257, 640), (64, 4160, 4096), (17, 100, 16),
                                   (64, 1000, 1536)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gemm_few_rows(M, N, K, dtype):
    gemm_case(M, N, K, dtype, M + N + K)


@pytest.mark.parametrize("M,N,K", [(65, 1, 1), (128, 192, 128), (129, 193, 260), (200, 130, 1000), (1001, 448, 1536),
                                   (333, 4160, 528), (2500, 1000, 272)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gemm_many_rows(M, N, K, dtype):
    gemm_case(M, N, K, dtype, M + N + K)


@pytest.mark.parametrize("M", [5, 150])
def test_gemm_strides_and_extreme_scales(M):
    gemm_case(M, 330, 700, F32, 1, spread=60, pad=3)


@pytest.mark.parametrize("M,N,K,pad,shift", [(301, 481, 144, 1, 0), (130, 480, 256, 0, 1), (200, 720, 128, 3, 5),
                                             (97, 239, 400, 0, 3), (256, 241, 128, 7, 0)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gemm_outputs_off_the_16_byte_grid(M, N, K, pad, shift, dtype):
    gemm_case(M, N, K, dtype, M + N + K, pad=pad, shift=shift)


# ---------------------------------------------------------------- attention
def entries(rng, n, c, spread=2):
    codes = rng.integers(0, 256, (n, c)).astype(np.uint8)
    codes[(codes & 127) > 0x70] &= 0x8F              # magnitudes below 16 mostly: scores of ordinary size
    return torch.as_tensor(codes).to(DEV), torch.as_tensor(rng.integers(118 - spread, 119 + spread, n).astype(np.uint8)).to(DEV)


def check_rows(dims, q, codes, scales, idx, base, avail, out, rows=None):
    nh, c = dims.nh, dims.c
    dtype = out.dtype
    worst = 0.0
    for r in rows if rows is not None else range(q.shape[0]):
        i = idx[r]
        sel = base[r] + i[(i >= 0) & (i < avail[r])].long().to(DEV)
        want, bound = ref.mqa(q[r, :nh * c].double().view(nh, c), codes, scales, sel, dtype)
        err = (out[r].double().view(nh, c) - want).abs()
        assert (err <= bound).all(), (r, float((err / bound.clamp(min=1e-30)).max()))
        worst = max(worst, float((err / bound.clamp(min=1e-30)).max()))
    return worst


def decode_mqa(dims, B, cap, avail, idx, seed, ld_pad=0, codes=None, scales=None, q=None):
    rng = np.random.default_rng(seed)
    if codes is None:
        codes, scales = entries(rng, B * cap, dims.c)
    dtype = BF16 if dims.dtype == csa.CSA_BF16 else F32
    w = dims.nh * dims.c
    if q is None:
        q = torch.as_tensor(rng.standard_normal((B, w + ld_pad)), dtype=F32).to(dtype).to(DEV)
    pos = torch.as_tensor([dims.m * a + min(1, dims.m - 1) for a in avail], dtype=torch.int32, device=DEV)
    out = torch.full((B, w), 9.0, dtype=dtype, device=DEV)
    ws = torch.empty(csa.csa_mqa_f8_workspace_bytes(dims, B), dtype=torch.uint8, device=DEV)
    csa.csa_decode_mqa_f8(dims, q, w + ld_pad, codes, scales, idx.to(DEV), pos, cap, B, out, ws)
    return q, codes, scales, out


def picked(rng, B, k, avail):
    idx = torch.full((B, k), -1, dtype=torch.int32)
    for b in range(B):
        n = min(k, avail[b])
        idx[b, :n] = torch.as_tensor(np.sort(rng.permutation(avail[b])[:n]).astype(np.int32))
    return idx


def tc_dims(nh, k, m=4):
    return csa.Dims(d=256, c=512, m=m, cI=128, nhI=64, nh=nh, dc=128, topk=k, dtype=csa.CSA_BF16)


@pytest.mark.parametrize("B,nh,k,cap", [(1, 64, 1, 5), (1, 64, 64, 80), (2, 64, 128, 200), (3, 128, 129, 300),
                                        (1, 128, 300, 310), (5, 64, 257, 700), (1, 128, 2048, 2500), (80, 128, 130, 140),
                                        (160, 64, 65, 90), (2, 192, 70, 100), (1, 192, 8192, 8300)])
def test_decode_mqa_tensor_cores(B, nh, k, cap):
    rng = np.random.default_rng(k + B)
    dims = tc_dims(nh, k)
    avail = [int(rng.integers(0, cap + 1)) for _ in range(B)]
    avail[0] = cap
    if B > 2:
        avail[1], avail[2] = 0, 1
    idx = picked(rng, B, k, avail)
    q, codes, scales, out = decode_mqa(dims, B, cap, avail, idx, k)
    assert csa.csa_get_device_status() == 0
    check_rows(dims, q, codes, scales, idx, [b * cap for b in range(B)], avail, out, range(min(B, 12)))


@pytest.mark.parametrize("dims", [
    csa.Dims(d=64, c=64, m=4, cI=32, nhI=4, nh=3, dc=64, topk=20, dtype=csa.CSA_BF16),
    csa.Dims(d=64, c=128, m=2, cI=32, nhI=4, nh=8, dc=64, topk=7, dtype=csa.CSA_F32),
    csa.Dims(d=64, c=256, m=1, cI=32, nhI=4, nh=5, dc=64, topk=33, dtype=csa.CSA_BF16),
    csa.Dims(d=64, c=512, m=8, cI=32, nhI=4, nh=64, dc=64, topk=40, dtype=csa.CSA_F32),
    csa.Dims(d=64, c=512, m=4, cI=32, nhI=4, nh=20, dc=64, topk=40, dtype=csa.CSA_BF16),
    csa.Dims(d=64, c=1024, m=4, cI=32, nhI=4, nh=2, dc=64, topk=9, dtype=csa.CSA_BF16),
])
def test_decode_mqa_other_configurations(dims):
    rng = np.random.default_rng(dims.c + dims.nh)
    B, cap = 4, 60
    avail = [60, 0, 1, 33]
    idx = picked(rng, B, dims.topk, avail)
    q, codes, scales, out = decode_mqa(dims, B, cap, avail, idx, 5, ld_pad=16)
    assert csa.csa_get_device_status() == 0
    check_rows(dims, q, codes, scales, idx, [b * cap for b in range(B)], avail, out)


@pytest.mark.parametrize("nh,B", [(64, 1), (64, 200), (128, 6)])
def test_decode_mqa_gaps_and_empty_rows(nh, B):
    """Valid slots scattered among -1 ones (whole tiles of them empty), rows without any."""
    rng = np.random.default_rng(11)
    k, cap = 700, 900
    dims = tc_dims(nh, k)
    avail = [cap] * B
    idx = torch.full((B, k), -1, dtype=torch.int32)
    for b in range(B):
        at = np.sort(rng.permutation(k)[:[40, 0, 1, 300][b % 4]])
        if b % 4 == 0:
            at = at[(at < 100) | (at >= 520)]        # tiles in the middle without a valid slot
        idx[b, at] = torch.as_tensor(np.sort(rng.permutation(cap)[:len(at)]).astype(np.int32))
    q, codes, scales, out = decode_mqa(dims, B, cap, avail, idx, 12, ld_pad=64)
    assert csa.csa_get_device_status() == 0
    check_rows(dims, q, codes, scales, idx, [b * cap for b in range(B)], avail, out, range(min(B, 8)))
    for b in range(B):
        if (idx[b] < 0).all():
            assert (out[b] == 0).all()


def test_decode_mqa_bad_index_is_flagged_and_skipped():
    rng = np.random.default_rng(13)
    dims = tc_dims(64, 40)
    avail = [50, 50]
    idx = picked(rng, 2, 40, avail)
    idx[0, 3], idx[1, 39] = 50, -7                    # beyond the visible entries; negative
    q, codes, scales, out = decode_mqa(dims, 2, 60, avail, idx, 14)
    assert csa.csa_get_device_status() == 5
    check_rows(dims, q, codes, scales, idx, [0, 60], avail, out)


def test_decode_mqa_bad_index_after_the_last_valid_slot_is_flagged():
    """Also where no part of the row is worked on: slots beyond the last valid one, and a row that sees nothing."""
    rng = np.random.default_rng(22)
    dims = tc_dims(64, 700)
    for avail, slot in ([60, 60], 650), ([60, 0], 3):
        idx = picked(rng, 2, 700, avail)
        idx[1, slot] = 60
        q, codes, scales, out = decode_mqa(dims, 2, 60, avail, idx, 23)
        assert csa.csa_get_device_status() == 5
        check_rows(dims, q, codes, scales, idx, [0, 60], avail, out)


@pytest.mark.parametrize("m", [1, 2, 8])
def test_decode_mqa_other_block_lengths(m):
    rng = np.random.default_rng(m)
    dims = tc_dims(64, 90, m)
    avail = [120, 0, 77]
    idx = picked(rng, 3, 90, avail)
    q, codes, scales, out = decode_mqa(dims, 3, 120, avail, idx, 24)
    assert csa.csa_get_device_status() == 0
    check_rows(dims, q, codes, scales, idx, [0, 120, 240], avail, out)


def test_decode_mqa_nan_stays_where_it_belongs():
    """NaN in one head's query, an infinite query value, NaN among one row's selected entries: NaN there, the other heads
    and rows right, the rows that the same CTA takes next among them."""
    rng = np.random.default_rng(25)
    B, cap = 300, 70
    dims = tc_dims(64, 66)
    idx = picked(rng, B, 66, [cap] * B)
    codes, scales = entries(rng, B * cap, 512)
    q = torch.as_tensor(rng.standard_normal((B, 64 * 512)), dtype=F32).to(BF16).to(DEV)
    q[299, 3 * 512 + 7] = float("nan")
    q[299, 5 * 512] = float("inf")
    q[298, 9 * 512 + 500] = float("-inf")
    codes[297 * cap + int(idx[297, 65]), 100] = 0x7F
    scales[296 * cap + int(idx[296, 0])] = 255
    q, codes, scales, out = decode_mqa(dims, B, cap, [cap] * B, idx, 26, codes=codes, scales=scales, q=q)
    assert csa.csa_get_device_status() == 0
    o = out.view(B, 64, 512)
    assert torch.isnan(o[299, [3, 5]]).all() and torch.isnan(o[298, 9]).all() and torch.isnan(o[296:298]).all()
    ok = torch.ones(B, 64, dtype=torch.bool)
    ok[299, [3, 5]] = ok[298, 9] = False
    ok[296:298] = False
    assert torch.isfinite(o[ok.to(DEV)]).all()
    check_rows(dims, q, codes, scales, idx, [b * cap for b in range(B)], [cap] * B, out, [0, 1, 148, 150, 151, 152, 295])
    for r in (298, 299):
        heads = ok[r].nonzero()[:, 0].to(DEV)
        want, bound = ref.mqa(q[r].double().view(64, 512)[heads], codes, scales, r * cap + idx[r].long().to(DEV), BF16)
        assert ((o[r][heads].double() - want).abs() <= bound).all()


def test_decode_mqa_unselected_rows_are_never_read():
    """NaN codes and NaN scales in every entry that no slot selects leave the output finite and right."""
    rng = np.random.default_rng(15)
    dims = tc_dims(64, 150)
    cap = 400
    idx = picked(rng, 1, 150, [cap])
    codes, scales = entries(rng, cap, 512)
    dead = torch.ones(cap, dtype=torch.bool)
    dead[idx[0].long()] = False
    codes[dead.to(DEV)] = 0x7F
    scales[dead.to(DEV)] = 255
    q, codes, scales, out = decode_mqa(dims, 1, cap, [cap], idx, 16, codes=codes, scales=scales)
    assert torch.isfinite(out).all()
    check_rows(dims, q, codes, scales, idx, [0], [cap], out)


@pytest.mark.parametrize("B", [1, 150])
def test_decode_mqa_growing_scores_and_unequal_scales(B):
    """Each tile's scores exceed the last one's (O is rescaled in flight), and entry scales differ by 2^40."""
    rng = np.random.default_rng(17)
    k = cap = 512
    dims = tc_dims(64, k)
    codes, scales = entries(rng, B * cap, 512)
    codes &= 0x7F                                     # positive: with q > 0 the scale orders the scores
    step = torch.arange(cap) // 128
    scales[:] = (100 + 9 * step).to(torch.uint8).repeat(B).to(DEV)
    scales[5], scales[200] = 140, 100
    q = torch.as_tensor(np.abs(rng.standard_normal((B, 64 * 512))), dtype=BF16).to(DEV)
    idx = torch.arange(cap, dtype=torch.int32).repeat(B, 1)
    q, codes, scales, out = decode_mqa(dims, B, cap, [cap] * B, idx, 18, codes=codes, scales=scales, q=q)
    assert csa.csa_get_device_status() == 0
    check_rows(dims, q, codes, scales, idx, [b * cap for b in range(B)], [cap] * B, out, range(min(B, 3)))


def test_decode_mqa_zero_entries_and_zero_queries():
    """Zero entries (scale byte 0) take part in the normaliser; a zero query averages its entries."""
    rng = np.random.default_rng(19)
    k = cap = 200
    dims = tc_dims(64, k)
    codes, scales = entries(rng, cap, 512)
    codes[::3] = 0
    scales[::3] = 0
    q = torch.as_tensor(rng.standard_normal((1, 64 * 512)), dtype=BF16).to(DEV)
    q[0, :512 * 5] = 0
    q[0, 512 * 5:512 * 6] *= 2.0 ** 60
    q[0, 512 * 6:512 * 7] *= 2.0 ** -60
    idx = torch.arange(cap, dtype=torch.int32)[None]
    q, codes, scales, out = decode_mqa(dims, 1, cap, [cap], idx, 20, codes=codes, scales=scales, q=q)
    rows = [h for h in range(64) if h != 5]           # head 5: scores of 2^60, a one-hot softmax
    want, bound = ref.mqa(q.double().view(64, 512), codes, scales, torch.arange(cap, device=DEV), BF16)
    err = (out.double().view(64, 512) - want).abs()
    assert (err[rows] <= bound[rows]).all()
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("lens,nh,k", [([300, 1, 3, 4, 517], 64, 33), ([2100], 64, 200), ([900, 700], 128, 512)])
def test_sparse_mqa_packed_rows(lens, nh, k):
    rng = np.random.default_rng(k)
    dims = tc_dims(nh, k)
    T = sum(lens)
    cu, cb = csa.cu_from_lengths(lens, dims.m)
    NB = int(cb[-1])
    codes, scales = entries(rng, NB, 512)
    q = torch.as_tensor(rng.standard_normal((T, nh * 512)), dtype=F32).to(BF16).to(DEV)
    base, avail = [], []
    for b, n in enumerate(lens):
        base += [int(cb[b])] * n
        avail += [t // dims.m for t in range(n)]
    idx = picked(rng, T, k, avail)
    out = torch.full((T, nh * 512), 9.0, dtype=BF16, device=DEV)
    ws = torch.empty(csa.csa_mqa_f8_workspace_bytes(dims, T), dtype=torch.uint8, device=DEV)
    csa.csa_sparse_mqa_f8(dims, q, nh * 512, codes, scales, idx.to(DEV), cu.to(DEV), cb.to(DEV), len(lens), T, NB, out,
                          ws)
    assert csa.csa_get_device_status() == 0
    some = sorted(set(rng.integers(0, T, 40).tolist()) | {0, 3, 4, T - 1, lens[0] - 1, min(lens[0], T - 1)})
    check_rows(dims, q, codes, scales, idx, base, avail, out, some)
