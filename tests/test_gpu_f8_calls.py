"""Calls of the 8-bit operators that their documentation allows: every number of K slices, packed rows so few that they
are split, an index named twice, weights that are not finite, decode steps queued one behind the other and replayed from
a graph."""
import numpy as np
import pytest
import torch

import compressed_sparse_attention_09_b200 as csa
import f8_ref as ref
from compressed_sparse_attention_09_b200 import synth
from test_gpu_f8 import BF16, DEV, F32, KIND, check_rows, decode_mqa, entries, gemm_case, picked, tc_dims
from test_gpu_f8_path import gemm_call, state
from test_gpu_parity import gpu_pack

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K,slices", [(64, 2304, 4096, 8), (1, 130, 4096, 8), (33, 4000, 2048, 1), (64, 9472, 1024, 1),
                                          (33, 4000, 4096, 4), (7, 4500, 8176, 4), (7, 4865, 4080, 1), (1, 4160, 3968, 1), (64, 4160, 4224, 1),
                                          (64, 520, 1536, 1), (5, 520, 2560, 1)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_product_by_slices(M, N, K, slices, dtype):
    """Eight and four slices (whole blocks at their ends or not) and sizes that are not sliced."""
    need = csa.csa_gemm_f8_workspace_bytes(M, N, K)
    assert need == (0 if slices == 1 else -(-slices * -(-N // 128) * 128 * M * 4 // 256) * 256)
    gemm_case(M, N, K, dtype, M + N + K)


@pytest.mark.parametrize("lens,nh,k", [([40, 1, 3, 20], 64, 9), ([65], 64, 70), ([17, 18], 128, 200), ([5], 192, 130)])
def test_few_packed_rows(lens, nh, k):
    """Packed rows that leave SMs idle are split like decode rows, those that see nothing yet among them."""
    rng = np.random.default_rng(k)
    dims = tc_dims(nh, k)
    T = sum(lens)
    cu, cb = csa.cu_from_lengths(lens, dims.m)
    NB = int(cb[-1])
    codes, scales = entries(rng, max(NB, 1), 512)
    q = torch.as_tensor(rng.standard_normal((T, nh * 512)), dtype=F32).to(BF16).to(DEV)
    base = [int(cb[b]) for b, n in enumerate(lens) for _ in range(n)]
    avail = [t // dims.m for n in lens for t in range(n)]
    idx = picked(rng, T, k, avail)
    out = torch.full((T, nh * 512), 9.0, dtype=BF16, device=DEV)
    ws = torch.empty(csa.csa_mqa_f8_workspace_bytes(dims, T), dtype=torch.uint8, device=DEV)
    csa.csa_sparse_mqa_f8(dims, q, nh * 512, codes, scales, idx.to(DEV), cu.to(DEV), cb.to(DEV), len(lens), T, NB, out, ws)
    assert csa.csa_get_device_status() == 0
    check_rows(dims, q, codes, scales, idx, base, avail, out)


@pytest.mark.parametrize("nh,B", [(64, 1), (64, 150), (20, 2)])
def test_an_index_named_twice_counts_twice(nh, B):
    rng = np.random.default_rng(nh + B)
    cap, k = 90, 140
    dims = tc_dims(nh, k)
    idx = torch.as_tensor(rng.integers(0, cap, (B, k)).astype(np.int32))
    idx[0] = 7                                        # one entry, k times
    q, codes, scales, out = decode_mqa(dims, B, cap, [cap] * B, idx, 3)
    assert csa.csa_get_device_status() == 0
    check_rows(dims, q, codes, scales, idx, [b * cap for b in range(B)], [cap] * B, out, range(min(B, 3)))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_weights_that_are_not_finite(dtype):
    """Infinite and NaN weights become NaN codes and leave their square's scale alone; a square without a finite value
    other than zero has byte 0."""
    rng = np.random.default_rng(4)
    N, K = 260, 400
    x = torch.as_tensor(rng.standard_normal((N, K)), dtype=F32).to(dtype)
    x[5, 3], x[127, 127], x[130, 260:264], x[259, 399] = float("inf"), float("-inf"), float("nan"), float("nan")
    x[128:256, 0:128] = float("-inf")
    x[256:, 384:] = float("nan")
    codes = torch.zeros(N, K, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(3, 4, dtype=torch.uint8, device=DEV)
    csa.csa_quantize_weight_f8(KIND[dtype], x.to(DEV), K, N, K, codes, K, scales, 4)
    assert csa.csa_get_device_status() == 0
    fin = torch.isfinite(x)
    want, ws = ref.quantize_squares(torch.where(fin, x, 0).double().numpy())
    codes = codes.cpu()
    assert np.array_equal(codes[fin].numpy(), want[fin.numpy()])
    assert ((codes[~fin] & 0x7F) == 0x7F).all()
    assert np.array_equal(scales.cpu().numpy(), ws) and ws[1, 0] == 0 and ws[2, 3] == 0


def test_sliced_products_captured_and_on_two_streams():
    """Two products in slices, each with its own workspace, replayed from graphs and queued on streams of their own."""
    calls = [gemm_call(7, 300, 4096, 1), gemm_call(64, 4160, 4096, 2)]
    assert csa.csa_gemm_f8_workspace_bytes(7, 300, 4096) and csa.csa_gemm_f8_workspace_bytes(64, 4160, 4096)
    want = []
    for call, v in calls:
        call()
        torch.cuda.synchronize()
        want.append(v["out"].clone())
        v["out"].zero_()
    streams = [torch.cuda.Stream() for _ in calls]
    graphs = []
    torch.cuda.synchronize()
    for (call, _), st in zip(calls, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            call()
        graphs.append(g)
    for how in "queued", "replayed":
        for _ in range(5):
            for (call, _), g, st in zip(calls, graphs, streams):
                if how == "queued":
                    call(st)
                else:
                    with torch.cuda.stream(st):
                        g.replay()
        torch.cuda.synchronize()
        assert csa.csa_get_device_status() == 0
        for (_, v), w in zip(calls, want):
            assert w.abs().sum() > 0 and torch.equal(v["out"], w), how
            v["out"].zero_()
        torch.cuda.synchronize()


# ---------------------------------------------------------------- the decode step, step behind step
def steps_state(B, nh, seed, cap):
    dims = csa.Dims(d=256, c=512, m=4, cI=128, nhI=64, nh=nh, dc=128, topk=100, dtype=csa.CSA_BF16)
    packed = gpu_pack(dims, synth.make_weights(dims, seed))
    packed8 = torch.empty(csa.csa_packed_weights_f8_bytes(dims), dtype=torch.uint8, device=DEV)
    csa.csa_pack_weights_f8(dims, packed, packed8)
    ws = torch.empty(csa.csa_decode_f8_workspace_bytes(dims, B, cap), dtype=torch.uint8, device=DEV)
    return dims, packed, packed8, ws


def step(dims, packed, packed8, ws, s, h, pos, O, cap, B, stream=None):
    csa.csa_decode_f8(dims, packed, packed8, h, pos, s["ring"], s["Cq"], s["Cs"], s["Kq"], s["Ks"], s["clen"], cap, B, O, None, ws,
                      stream)


@pytest.mark.parametrize("B,nh", [(1, 128), (3, 64), (70, 64)])
def test_decode_steps_queued_and_replayed(B, nh):
    """Nine steps (two appends and more), each waited for; queued one behind the other; and replayed from one captured
    step whose inputs are copied in: the same outputs, caches and rings to the bit."""
    pos0, cap, n = 201, 64, 9
    dims, packed, packed8, ws = steps_state(B, nh, 40, cap)
    first = state(dims, B, cap, pos0, 41)
    h = [synth.make_normal((B, dims.d), dims, 60 + i).to(DEV) for i in range(n)]
    pos = [torch.full((B,), pos0 + i, dtype=torch.int32, device=DEV) for i in range(n)]
    new = lambda: [torch.zeros(B, nh * 512, dtype=BF16, device=DEV) for _ in range(n)]   # noqa: E731

    waited, queued, replayed = new(), new(), new()
    s1 = {k: v.clone() for k, v in first.items()}
    for i in range(n):
        step(dims, packed, packed8, ws, s1, h[i], pos[i], waited[i], cap, B)
        assert csa.csa_get_device_status() == 0       # (synchronises)
    s2 = {k: v.clone() for k, v in first.items()}
    torch.cuda.synchronize()
    for i in range(n):
        step(dims, packed, packed8, ws, s2, h[i], pos[i], queued[i], cap, B)
    torch.cuda.synchronize()

    s3 = {k: v.clone() for k, v in first.items()}
    gh, gpos, gO = h[0].clone(), pos[0].clone(), torch.zeros_like(replayed[0])
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        step(dims, packed, packed8, ws, s3, gh, gpos, gO, cap, B)
    for i in range(n):
        gh.copy_(h[i])
        gpos.copy_(pos[i])
        graph.replay()
        replayed[i].copy_(gO)
    torch.cuda.synchronize()
    assert csa.csa_get_device_status() == 0
    for i in range(n):
        assert torch.isfinite(waited[i]).all() and waited[i].abs().sum() > 0
        assert torch.equal(waited[i], queued[i]) and torch.equal(waited[i], replayed[i]), i
    for k in first:
        assert torch.equal(s1[k], s2[k]) and torch.equal(s1[k], s3[k]), k


def test_the_attention_repeats_itself():
    """The same inputs give the same bits, call after call."""
    rng = np.random.default_rng(2)
    for nh, B, cap in (128, 1, 700), (128, 64, 300), (64, 200, 200):
        dims = tc_dims(nh, cap)
        idx = picked(rng, B, cap, [cap] * B)
        q, codes, scales, out = decode_mqa(dims, B, cap, [cap] * B, idx, 5)
        for _ in range(20):
            again = decode_mqa(dims, B, cap, [cap] * B, idx, 5, codes=codes, scales=scales, q=q)[3]
            assert torch.equal(out, again), (nh, B)
    assert csa.csa_get_device_status() == 0
