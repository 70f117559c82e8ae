"""The grouped linear where every pipeline runs on: clusters and CTAs with several tiles, reductions
longer than the stages, tiles of two MMAs, more than 32 waves, warps with several rows.

On a GPU of 152 SMs the products have 76 clusters, 4 stages of 256 along the reduction (7 for few tokens),
tiles of up to 384 columns and find their tiles 32 waves at a time; the quantizers have 304 CTAs with
rings of 3 tiles, the row-blob kernel 4864 warps.  Products equal the library's single GEMM bit for
bit, group by group: both sum along the reduction in the same order.  Blobs equal the oracle's byte for byte.
"""
import numpy as np
import pytest
import torch

import oracle
from mxfp4_block_scaled_quantize_gb300 import abi, workloads
from mxfp4_block_scaled_quantize_gb300.grouped import MXFP4GroupedLinear
from parity import check_gemm
from test_gpu_grouped import check_blobs, check_products, offsets_of, products, routing

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert abi.mxfp4_last_device_error() == abi.MXFP4_OK


def ragged(groups, total, seed, empty=0.15):
    """Group sizes that sum to `total`: uneven, some empty, some of one row."""
    rng = np.random.default_rng(seed)
    share = rng.exponential(1.0, groups) * (rng.random(groups) >= empty)
    counts = np.floor(share / share.sum() * (total - 2)).astype(int)
    counts[rng.integers(groups)] += total - counts.sum()
    return counts.tolist()


def step_against_the_single_gemm(counts, N, K, dtype, gathered, seed=0):
    """A layer's step, each group's products against the plain quantizer and GEMM."""
    E, R = len(counts), sum(counts)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *shape: torch.randn(*shape, generator=gen, device="cuda").to(torch.bfloat16)
    T = max(R // 3, 1) if gathered else R
    x, w, dy = rnd(T, K), rnd(E, N, K), rnd(R, N)
    idx = torch.randint(0, T, (R,), generator=gen, device="cuda", dtype=torch.int32) if gathered else None
    od, o = offsets_of(counts)
    layer = MXFP4GroupedLinear(E, N, K, R, out_dtype=dtype)
    y, dx, dw = layer.step(x, w, dy, od, idx)
    torch.cuda.synchronize()
    assert abi.mxfp4_last_device_error() == abi.MXFP4_OK
    g = x if idx is None else x[idx.long()]
    for e, c in enumerate(counts):
        if c == 0:
            assert torch.count_nonzero(dw[e]) == 0, f"dw of empty group {e}"
            continue
        rows = slice(int(o[e]), int(o[e + 1]))
        xq, wq, dq = (abi.quantize(t.contiguous()) for t in (g[rows], w[e], dy[rows]))
        for got, want, name in ((y[rows], abi.gemm(*xq[:2], *wq[:2], c, N, K, out_dtype=dtype), "y"),
                                (dx[rows], abi.gemm(*dq[:2], *wq[2:], c, K, N, out_dtype=dtype), "dx"),
                                (dw[e], abi.gemm(*dq[2:], *xq[2:], N, K, c, out_dtype=dtype), "dw")):
            assert torch.equal(got, want), f"{name} of group {e} with {c} rows"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gathered", [True, False])
def test_many_tiles_a_cluster_and_long_reductions(gathered, dtype):
    # 8 strips of W times some 25 token tiles, 8 steps along K; wgrad 16 x 8 x 6 tiles, groups of up to
    # 1500 rows; X and W quantized apart (16 tiles a CTA)
    step_against_the_single_gemm(ragged(16, 5000, 1), 2048, 2048, dtype, gathered)


@pytest.mark.parametrize("sizes", [(5, 1500, 1032, 1416), (8, 2048, 1536, 1536), (3, 4000, 200, 3000)])
def test_x_and_w_in_one_launch_with_several_tiles_a_cta(sizes):
    E, R, N, K = sizes
    step_against_the_single_gemm(ragged(E, R, 2, empty=0), N, K, torch.bfloat16, True, seed=1)
    step_against_the_single_gemm(ragged(E, R, 3, empty=0), N, K, torch.bfloat16, False, seed=2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_few_tokens_and_a_long_reduction(dtype):
    # the instance for few tokens: 7 stages, 16 steps; 16 strips of W for each of 64 groups
    step_against_the_single_gemm(ragged(64, 1500, 4), 4096, 4096, dtype, True)


def test_one_large_group_among_small_ones():
    # 47 tiles of 128 tokens in the instance for few tokens, which goes by the average
    counts = [1] * 64
    counts[40] = 5900
    step_against_the_single_gemm(counts, 512, 1024, torch.bfloat16, True)


@pytest.mark.parametrize("rows", [3000, 110000])
def test_more_than_32_waves(rows):
    # 1024 groups of 3 strips: 3072 tiles and more for 76 clusters, with few tokens and with many
    step_against_the_single_gemm(ragged(1024, rows, 5), 768, 256, torch.bfloat16, rows < 10000)


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_tiles_of_two_mmas_against_the_oracle(out_dtype):
    counts, N, K = [130, 0, 1, 384, 700, 385, 289], 264, 1352
    got, cpu, o = products(counts, N, K, out_dtype, seed=6)
    check_products(got, cpu, o, counts, N, K, "two MMAs")


# ---------------------------------------------------------------------------------------
# quantizers
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("gathered", [True, False])
@pytest.mark.parametrize("dual", [True, False])
@pytest.mark.parametrize("K", [2048, 1544])
def test_quantizers_with_several_tiles_a_cta(K, dual, gathered):
    # 80 row tiles and more x 16 (13): 4 tiles and more a CTA; rows of 2 pieces: 3 pieces a warp
    counts = ragged(64, 7000, 7)
    R, T = sum(counts), 2500 if gathered else 7000
    x = workloads.student_t3((T, K), 1.0, 30 + K)
    od, o = offsets_of(counts)
    idx = torch.randint(0, T, (R,), generator=torch.Generator().manual_seed(K), dtype=torch.int32) if gathered else None
    bits = workloads.bf16_bits(x)
    blobs = abi.quantize_grouped(x.cuda(), od, None if idx is None else idx.cuda(), dual=dual)
    check_blobs(blobs, bits if idx is None else bits[idx.numpy()], o, counts,
                abi.mxfp4_grouped_sizes(R, K, len(counts))[4], f"K={K} {dual} {gathered}")


@pytest.mark.parametrize("gathered", [True, False])
def test_row_blob_with_many_rows_a_warp(gathered):
    # 41 rows of one piece a warp: the indices are fetched again after 32, and groups end inside a warp's run
    counts, K = ragged(300, 200000, 8), 40
    R, T = sum(counts), 900 if gathered else 200000
    x = workloads.normal((T, K), 1.0, 31)
    od, o = offsets_of(counts)
    idx = torch.randint(0, T, (R,), generator=torch.Generator().manual_seed(9), dtype=torch.int32) if gathered else None
    bits = workloads.bf16_bits(x)
    blobs = abi.quantize_grouped(x.cuda(), od, None if idx is None else idx.cuda(), dual=False)
    check_blobs(blobs, bits if idx is None else bits[idx.numpy()], o, counts,
                abi.mxfp4_grouped_sizes(R, K, len(counts))[4], f"many rows {gathered}")


# ---------------------------------------------------------------------------------------
# serving
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens", [1, 24, 700])
def test_packed_weights_against_the_oracle(tokens, out_dtype):
    E, N, K = 6, 272, 1352
    w = workloads.normal((E, N, K), 0.02, 41)
    bits = workloads.bf16_bits(w.view(-1, K))
    w_q, w_s = abi.quantize_grouped(w.view(-1, K).cuda(), groups=E, dual=False)
    idx, counts = routing(tokens, E, 2, tokens)
    od, o = offsets_of(counts)
    x = workloads.normal((tokens, K), 1.0, 42)
    g = workloads.bf16_bits(x)[idx.cpu().numpy()]
    want = [None if c == 0 else oracle.gemm(*oracle.quantize_row(np.ascontiguousarray(g[o[e]:o[e + 1]])),
                                            *oracle.quantize_row(np.ascontiguousarray(bits[e * N:(e + 1) * N])))
            for e, c in enumerate(counts)]

    def check(y, what):
        for e, pair in enumerate(want):
            if pair is not None:
                check_gemm(y[int(o[e]):int(o[e + 1])], *pair, f"{what} expert {e}")

    xg = x.cuda()
    layer = MXFP4GroupedLinear(E, N, K, 2 * tokens, train=False, out_dtype=out_dtype)
    check(layer.forward_packed(xg, w_q, w_s, od, idx), "eager")
    layer.y.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = layer.forward_packed(xg, w_q, w_s, od, idx)
    side.synchronize()
    check(y, "another stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer.forward_packed(xg, w_q, w_s, od, idx)
    layer.y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    check(y, "graph")


def test_one_row_whatever_its_stride():
    # a column turned round is a row of K elements whose row stride is 1
    E, N, K = 2, 136, 264
    w = workloads.normal((E, N, K), 0.02, 51).cuda()
    x, dy = workloads.normal((K, 1), 1.0, 52).cuda().t(), workloads.normal((N, 1), 1.0, 53).cuda().t()
    od, _ = offsets_of([0, 1])
    layer = MXFP4GroupedLinear(E, N, K, 1)
    got = [t.clone() for t in layer.step(x, w, dy, od)]
    plain = layer.step(x.clone(memory_format=torch.contiguous_format).view(-1).view(1, K), w, dy.reshape(-1).view(1, N), od)
    for a, b in zip(got, plain):
        assert torch.equal(a, b)
    for blobs in (abi.quantize_grouped(x, od), abi.quantize_grouped(x, groups=1)):
        assert torch.equal(blobs[0], abi.quantize(x.reshape(-1).view(1, K))[0])
