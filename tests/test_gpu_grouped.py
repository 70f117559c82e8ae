"""GPU parity of the grouped MXFP4 linear (ragged groups whose sizes only the device knows).

Blobs: bit-exact against the oracle's quantization of the gathered rows (row blob) and of the
group-padded matrix (col blob).  Products: the GEMM's own accuracy contract (parity.check_gemm)
against fp64 sums of the oracle's dequantized blobs, group by group, and bit for bit equal to
the library's single GEMM on the same rows.
"""
import numpy as np
import pytest
import torch

import oracle
from mxfp4_block_scaled_quantize_gb300 import abi, workloads
from mxfp4_block_scaled_quantize_gb300.grouped import MXFP4GroupedLinear
from parity import assert_bytes_equal, check_gemm, tc_index

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert abi.mxfp4_last_device_error() == abi.MXFP4_OK


def pitched(x_cpu):
    """CUDA copy of x with a row pitch rounded up to a multiple of 8 elements."""
    M, K = x_cpu.shape
    wide = torch.full((M, (K + 7) // 8 * 8), float("nan"), dtype=x_cpu.dtype, device="cuda")
    wide[:, :K] = x_cpu.cuda()
    return wide[:, :K]


def offsets_of(counts, first=0):
    o = np.concatenate([[0], np.cumsum(counts)]) + first
    return torch.tensor(o, dtype=torch.int32, device="cuda"), o


def padded_rows(counts):
    """Padded row of each group's start, and the end of the last."""
    return np.concatenate([[0], np.cumsum([(c + 127) // 128 * 128 for c in counts])])


def padded_bits(bits, o, counts):
    """The group-padded matrix that the col blob describes."""
    P = padded_rows(counts)
    out = np.zeros((P[-1], bits.shape[1]), np.uint16)
    for e, c in enumerate(counts):
        out[P[e]:P[e] + c] = bits[o[e]:o[e + 1]]
    return out


def tc_rows(s, rows, KB):
    rr, kk = np.meshgrid(rows, np.arange(KB), indexing="ij")
    return s.cpu().numpy()[tc_index(rr, kk, KB)]


def check_blobs(blobs, bits, o, counts, capacity, what):
    """Every byte that a grouped blob defines: bits = the bf16 patterns of G."""
    K, dual = bits.shape[1], len(blobs) == 4
    live = np.arange(o[0], o[-1])
    if live.size == 0:
        return
    rq, rs = oracle.quantize_row(np.ascontiguousarray(bits[live]))
    assert_bytes_equal(blobs[0].cpu().numpy()[live], rq, f"{what} row q")
    P = padded_rows(counts)
    at = np.concatenate([P[e] + np.arange(c) for e, c in enumerate(counts)]).astype(np.int64)
    assert_bytes_equal(tc_rows(blobs[1], at, rs.shape[1]), rs, f"{what} row s")
    if dual:
        cq, cs = oracle.quantize_col(padded_bits(bits, o, counts))
        assert_bytes_equal(blobs[2].cpu().numpy()[:, :P[-1] // 2], cq, f"{what} col q")
        kp = (K + 127) // 128 * 128
        got = tc_rows(blobs[3], np.arange(kp), capacity // 32)[:, :P[-1] // 32]
        want = np.zeros((kp, cs.shape[1]), np.uint8)   # padding rows of the layout: 0x00
        want[:K] = cs
        assert_bytes_equal(got, want, f"{what} col s")


COUNTS = {
    "one_row": [1],
    "empty_ends": [0, 1, 0],
    "decode": [1, 0, 2, 0, 0, 1, 1, 3],
    "tile_edges": [127, 128, 129, 0, 255, 256, 257],
    "ragged": [5, 300, 0, 64, 33, 1, 700],
}


@pytest.mark.parametrize("K", [8, 32, 100, 128, 257, 1032])
@pytest.mark.parametrize("name", sorted(COUNTS))
def test_quantize_grouped_bytes(name, K):
    counts = COUNTS[name]
    R = sum(counts)
    T = max(3, R // 2)
    x = workloads.student_t3((T, K), 1.0, 11 + K)
    idx = torch.randint(0, T, (R,), generator=torch.Generator().manual_seed(K), dtype=torch.int32)
    od, o = offsets_of(counts)
    bits = workloads.bf16_bits(x)[idx.numpy()]
    xg = pitched(x)
    cap = abi.mxfp4_grouped_sizes(R, K, len(counts))[4]
    for dual in (False, True):
        check_blobs(abi.quantize_grouped(xg, od, idx.cuda(), dual=dual), bits, o, counts, cap, f"{name} K={K} {dual}")


def test_quantize_grouped_special_values_and_no_index():
    counts, K = [40, 0, 130, 7], 160
    x = workloads.inject_edge_blocks(workloads.student_t3((sum(counts), K), 1e-4, 3), 5)
    od, o = offsets_of(counts)
    bits = workloads.bf16_bits(x)
    cap = abi.mxfp4_grouped_sizes(sum(counts), K, len(counts))[4]
    for dual in (False, True):
        check_blobs(abi.quantize_grouped(x.cuda(), od, dual=dual), bits, o, counts, cap, f"edges {dual}")


def test_quantize_equal_groups_are_the_plain_blobs():
    # offsets None: groups of equal size; a size of whole tiles makes the blobs the plain quantizer's
    E, n, K = 3, 256, 192
    x = workloads.normal((E * n, K), 1.0, 7).cuda()
    for got, want in zip(abi.quantize_grouped(x, groups=E), abi.quantize(x, dual=True)):
        assert torch.equal(got.view(-1), want.view(-1))
    # and 200 rows a group are padded to 256 each
    counts, o = [200] * E, np.arange(E + 1) * 200
    x = workloads.normal((E * 200, K), 1.0, 8)
    check_blobs(abi.quantize_grouped(x.cuda(), groups=E), workloads.bf16_bits(x), o, counts, E * 256, "equal 200")


def test_most_groups_and_rows_outside_every_group():
    counts = [0] * 1024
    for e, c in ((0, 1), (31, 2), (32, 130), (33, 1), (700, 129), (1023, 3)):
        counts[e] = c
    R, K, first = sum(counts) + 9, 96, 4   # 4 rows before the first group, 5 after the last
    x = workloads.normal((R, K), 1.0, 9)
    od, o = offsets_of(counts, first)
    cap = abi.mxfp4_grouped_sizes(R, K, 1024)[4]
    for dual in (False, True):
        check_blobs(abi.quantize_grouped(x.cuda(), od, rows=R, dual=dual), workloads.bf16_bits(x), o, counts, cap, "1024")


def products(counts, N, K, out_dtype, seed=0, ldc_pad=0, first=0, tail=0):
    """The three products on the GPU (outputs pre-filled with 7) and the bf16 operands on the CPU."""
    E, R = len(counts), sum(counts) + first + tail
    od, o = offsets_of(counts, first)
    x = workloads.normal((R, K), 1.0, 100 + seed)
    w = workloads.normal((E * N, K), 0.02, 101 + seed)
    dy = workloads.normal((R, N), 1e-3, 102 + seed)
    xb = abi.quantize_grouped(pitched(x), od, rows=R)
    wb = abi.quantize_grouped(pitched(w), groups=E)
    db = abi.quantize_grouped(pitched(dy), od, rows=R)
    code = abi.MXFP4_OUT_F32 if out_dtype == torch.float32 else abi.MXFP4_OUT_BF16

    def out(rows, cols):
        return torch.full((rows, cols + ldc_pad), 7.0, dtype=out_dtype, device="cuda")

    y, dx, dw = out(R, N), out(R, K), out(E * N, K)
    abi.mxfp4_gemm_grouped(abi.MXFP4_GROUPED_FWD, *xb[:2], *wb[:2], od, E, R, N, K, y, y.stride(0), code)
    abi.mxfp4_gemm_grouped(abi.MXFP4_GROUPED_DGRAD, *db[:2], *wb[2:], od, E, R, N, K, dx, dx.stride(0), code)
    abi.mxfp4_gemm_grouped(abi.MXFP4_GROUPED_WGRAD, *db[2:], *xb[2:], od, E, R, N, K, dw, dw.stride(0), code)
    torch.cuda.synchronize()
    assert abi.mxfp4_last_device_error() == abi.MXFP4_OK
    return (y, dx, dw), (x, w, dy), o


def check_products(got, cpu, o, counts, N, K, what):
    (y, dx, dw), (x, w, dy) = got, cpu
    xb, wb, db = (workloads.bf16_bits(t) for t in (x, w, dy))
    for e, c in enumerate(counts):
        rows = slice(int(o[e]), int(o[e + 1]))
        dw_e = dw[e * N:(e + 1) * N]
        if c == 0:
            assert torch.count_nonzero(dw_e[:, :K]) == 0, f"{what} dw of empty group {e}"
            continue
        we = np.ascontiguousarray(wb[e * N:(e + 1) * N])
        xe, de = np.ascontiguousarray(xb[rows]), np.ascontiguousarray(db[rows])
        check_gemm(y[rows, :N], *oracle.gemm(*oracle.quantize_row(xe), *oracle.quantize_row(we)), f"{what} y[{e}]")
        check_gemm(dx[rows, :K], *oracle.gemm(*oracle.quantize_row(de), *oracle.quantize_col(we)), f"{what} dx[{e}]")
        check_gemm(dw_e[:, :K], *oracle.gemm(*oracle.quantize_col(de), *oracle.quantize_col(xe)), f"{what} dw[{e}]")


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,K", [(8, 8), (128, 128), (136, 264), (300, 520), (513, 97)])
@pytest.mark.parametrize("name", sorted(COUNTS))
def test_grouped_products(name, N, K, out_dtype):
    got, cpu, o = products(COUNTS[name], N, K, out_dtype)
    check_products(got, cpu, o, COUNTS[name], N, K, f"{name} {N}x{K}")


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_only_the_groups_rows_and_columns_are_written(out_dtype):
    # rows outside every group and the columns past the result's, inside the pitch, keep their value
    counts, N, K = [3, 0, 40, 130], 72, 136
    for pad in (8, 5):   # a pitch for tensor stores, and one for plain stores
        got, cpu, o = products(counts, N, K, out_dtype, ldc_pad=pad, first=6, tail=11)
        check_products(got, cpu, o, counts, N, K, f"pad {pad}")
        y, dx, dw = got
        for t, cols in ((y, N), (dx, K)):
            assert bool((t[:6] == 7).all()) and bool((t[-11:] == 7).all()) and bool((t[:, cols:] == 7).all())
        assert bool((dw[:, K:] == 7).all())


def test_products_equal_the_single_gemm_bit_for_bit():
    counts, N, K = [130, 0, 1, 512, 259], 384, 640
    (y, dx, dw), (x, w, dy), o = products(counts, N, K, torch.bfloat16, seed=5)
    for e, c in enumerate(counts):
        if c == 0:
            continue
        rows = slice(int(o[e]), int(o[e + 1]))
        xq, wq, dq = (abi.quantize(t.cuda().contiguous()) for t in (x[rows], w[e * N:(e + 1) * N], dy[rows]))
        assert torch.equal(y[rows], abi.gemm(*xq[:2], *wq[:2], c, N, K))
        assert torch.equal(dx[rows], abi.gemm(*dq[:2], *wq[2:], c, K, N))
        assert torch.equal(dw[e * N:(e + 1) * N], abi.gemm(*dq[2:], *xq[2:], N, K, c))


def test_no_rows_at_all():
    E, N, K = 3, 40, 48
    od, _ = offsets_of([0] * E)
    x = torch.empty((0, K), dtype=torch.bfloat16, device="cuda")
    blobs = abi.quantize_grouped(x, od)
    assert blobs[0].numel() == 0
    dw = torch.full((E * N, K), 7.0, device="cuda")
    wb = abi.quantize_grouped(workloads.normal((E * N, K), 1.0, 1).cuda(), groups=E)
    y = torch.empty((0, N), device="cuda")
    abi.mxfp4_gemm_grouped(abi.MXFP4_GROUPED_FWD, None, None, *wb[:2], od, E, 0, N, K, y, N, abi.MXFP4_OUT_F32)
    abi.mxfp4_gemm_grouped(abi.MXFP4_GROUPED_WGRAD, None, None, None, None, od, E, 0, N, K, dw, K, abi.MXFP4_OUT_F32)
    assert torch.count_nonzero(dw) == 0


def routing(T, E, k, seed):
    g = torch.Generator().manual_seed(seed)
    chosen = (torch.randn(T, E, generator=g) + torch.randn(E, generator=g)).topk(k, dim=1).indices.reshape(-1)
    order = torch.argsort(chosen, stable=True)
    counts = torch.bincount(chosen, minlength=E).tolist()
    return (order // k).to(torch.int32).cuda(), counts


def test_layer_step_and_reuse_with_fewer_rows():
    E, N, K, T = 6, 272, 392, 150
    layer = MXFP4GroupedLinear(E, N, K, 2 * T, out_dtype=torch.float32)
    w = workloads.normal((E, N, K), 0.02, 1)
    for seed, tokens in ((1, T), (2, 40), (3, T)):   # the same layer, another routing each step
        idx, counts = routing(tokens, E, 2, seed)
        od, o = offsets_of(counts)
        x = workloads.normal((tokens, K), 1.0, 10 + seed)
        dy = workloads.normal((2 * tokens, N), 1e-3, 20 + seed)
        y, dx, dw = layer.step(x.cuda(), w.cuda(), dy.cuda(), od, idx)
        check_products((y, dx, dw.view(-1, K)), (x[idx.cpu().long()], w.view(-1, K), dy), o, counts, N, K, f"step {seed}")


def test_serving_layer_on_another_stream_and_in_a_graph():
    E, N, K, T = 8, 256, 512, 24
    idx, counts = routing(T, E, 2, 4)
    od, o = offsets_of(counts)
    x, w = workloads.normal((T, K), 1.0, 5).cuda(), workloads.normal((E, N, K), 0.02, 6).cuda()
    layer = MXFP4GroupedLinear(E, N, K, 2 * T, train=False)
    layer.quantize_w(w)
    want = layer.forward(x, None, od, idx).clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer.y.zero_()
        got = layer.forward(x, None, od, idx).clone()
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer.forward(x, None, od, idx)
    # other tokens and another routing in the same buffers: the graph reads the sizes on the device
    idx2, counts2 = routing(T, E, 2, 44)
    x.copy_(workloads.normal((T, K), 1.0, 55))
    od.copy_(offsets_of(counts2)[0])
    idx.copy_(idx2)
    graph.replay()
    torch.cuda.synchronize()
    replayed = y.clone()
    assert torch.equal(replayed, layer.forward(x, None, od, idx))


def test_offsets_and_indices_out_of_range_are_recorded():
    # the library's own bounds checks: a bad index reads as a zero row, offsets are clamped
    K, N, E = 128, 128, 3
    x = workloads.normal((10, K), 1.0, 2)
    w = abi.quantize_grouped(workloads.normal((E * N, K), 1.0, 3).cuda(), groups=E)
    idx = torch.tensor([0, 10, -1, 2**30, 5, 9], dtype=torch.int32, device="cuda")
    od, o = offsets_of([2, 1, 3])
    blobs = abi.quantize_grouped(x.cuda(), od, idx)
    assert abi.mxfp4_last_device_error() == abi.MXFP4_ERR_GROUPS
    bits = workloads.bf16_bits(x)[[0, 0, 0, 0, 5, 9]]
    bits[1:4] = 0
    check_blobs(blobs, bits, o, [2, 1, 3], abi.mxfp4_grouped_sizes(6, K, E)[4], "bad index")
    for bad, counts in (([0, 4, 2, 6], [4, 0, 2]), ([-5, 3, 100, 6], [3, 3, 0]), ([2, 1, 0, -1], [0, 0, 0])):
        first = max(bad[0], 0)
        od = torch.tensor(bad, dtype=torch.int32, device="cuda")
        y = torch.full((6, N), 7.0, device="cuda")
        xb = abi.quantize_grouped(x.cuda()[:6], od)
        assert abi.mxfp4_last_device_error() == abi.MXFP4_ERR_GROUPS
        abi.mxfp4_gemm_grouped(abi.MXFP4_GROUPED_FWD, *xb[:2], *w[:2], od, E, 6, N, K, y, N, abi.MXFP4_OUT_F32)
        assert abi.mxfp4_last_device_error() == abi.MXFP4_ERR_GROUPS
        live = sum(counts)
        assert bool((y[:first] == 7).all()) and bool((y[first + live:] == 7).all())
        assert not bool((y[first:first + live] == 7).any())
    assert abi.mxfp4_last_device_error() == abi.MXFP4_OK
