"""Host-side checks of the grouped linear that need no GPU: sizes, refusals, and the group
table's arithmetic restated in Python."""
import ctypes

import pytest

from mxfp4_block_scaled_quantize_gb300 import abi


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return abi.load()


def test_capacity_holds_every_split(lib):
    import itertools
    for rows, groups in ((1, 1), (3, 2), (129, 2), (130, 3), (256, 3), (5, 4)):
        cap = abi.mxfp4_grouped_sizes(rows, 32, groups)[4]
        most = 0
        for cuts in itertools.combinations_with_replacement(range(rows + 1), groups - 1):
            edges = (0, *cuts, rows)
            most = max(most, sum((b - a + 127) // 128 * 128 for a, b in zip(edges, edges[1:])))
        assert most == cap, (rows, groups)   # enough for any split, and some split needs it


def test_sizes(lib):
    # 300 rows in 4 ragged groups: floor((300 + 127 * 4) / 128) = 6 tiles
    assert abi.mxfp4_grouped_sizes(300, 100, 4) == (300 * 64, 768 * 4, 100 * 384, 128 * 24, 768)
    # equal groups of 75 rows: one tile each
    assert abi.mxfp4_grouped_sizes(300, 100, 4, True)[4] == 512
    assert abi.mxfp4_grouped_sizes(0, 100, 4) == (0, 0, 0, 0, 0)
    for bad in ((-1, 8, 1, 0), (4, 0, 1, 0), (4, 8, 0, 0), (4, 8, 1025, 0), (5, 8, 2, 1), (2**31, 8, 1, 0)):
        with pytest.raises(abi.Mxfp4Error) as e:
            abi.mxfp4_grouped_sizes(*bad)
        assert e.value.status == abi.MXFP4_ERR_INVALID_ARG


def test_quantize_refusals(lib):
    bad, mis = abi.MXFP4_ERR_INVALID_ARG, abi.MXFP4_ERR_MISALIGNED
    # x, x_rows, K, ldx, row_index, offsets, groups, rows, q_row, s_row, q_col, s_col, stream
    ok = [16, 8, 8, 8, 32, 64, 2, 8, 48, 80, 96, 112, None]

    def call(**change):
        names = ["x", "x_rows", "K", "ldx", "row_index", "offsets", "groups", "rows", "q_row", "s_row", "q_col", "s_col"]
        a = list(ok)
        for k, v in change.items():
            a[names.index(k)] = v
        return lib.mxfp4_quantize_grouped(*a)

    assert call(x=None) == bad and call(q_row=None) == bad and call(s_row=None) == bad
    assert call(q_col=None) == bad and call(s_col=None) == bad          # both or neither
    assert call(K=0) == bad and call(ldx=0) == bad and call(rows=-1) == bad and call(x_rows=-1) == bad
    assert call(groups=0) == bad and call(groups=1025) == bad
    assert call(x_rows=0) == bad                                         # rows from nowhere
    assert call(row_index=None, x_rows=7) == bad                         # fewer rows than G without an index
    assert call(offsets=None, rows=7) == bad                             # equal groups of 3.5 rows
    assert call(x=24) == mis and call(ldx=12) == mis and call(q_row=40) == mis and call(s_row=88) == mis
    assert call(q_col=100) == mis and call(s_col=104) == mis and call(row_index=34) == mis and call(offsets=66) == mis


def test_gemm_refusals(lib):
    bad, mis = abi.MXFP4_ERR_INVALID_ARG, abi.MXFP4_ERR_MISALIGNED
    names = ["form", "a_q", "a_s", "b_q", "b_s", "offsets", "groups", "rows", "N", "K", "c", "ldc", "out_dtype"]
    ok = [0, 16, 32, 48, 64, 80, 2, 8, 8, 24, 96, 24, 0, None]

    def call(**change):
        a = list(ok)
        for k, v in change.items():
            a[names.index(k)] = v
        return lib.mxfp4_gemm_grouped(*a)

    assert call(form=3) == bad and call(form=-1) == bad
    for p in ("a_q", "a_s", "b_q", "b_s", "c"):
        assert call(**{p: None}) == bad and call(**{p: 24}) == mis
    assert call(groups=0) == bad and call(rows=-1) == bad and call(N=0) == bad and call(K=0) == bad
    assert call(ldc=7) == bad                        # forward: at least N
    assert call(form=1, ldc=23) == bad and call(form=2, ldc=23) == bad   # gradients: at least K
    assert call(out_dtype=2) == bad and call(offsets=82) == mis
    assert call(offsets=None, rows=7) == bad
    assert call(groups=1024, N=2**22) == bad         # more weight rows than coordinates
    assert call(form=2, rows=0, a_q=None, a_s=None, b_q=None, b_s=None, c=None) == bad


def layer_struct(**change):
    f = dict(groups=2, N=8, K=24, y=0x1000, dx=0x2000, dw=0x3000, out_dtype=0,
             x_blobs=(16, 32, 48, 64), w_blobs=(80, 96, 112, 128), dy_blobs=(144, 160, 176, 192))
    f.update(change)
    c = abi.GroupedLinear(**{k: v for k, v in f.items() if not k.endswith("blobs")})
    for name in ("x_blobs", "w_blobs", "dy_blobs"):
        getattr(c, name)[:] = f[name]
    return c


def test_layer_call_refusals(lib):
    bad, mis = abi.MXFP4_ERR_INVALID_ARG, abi.MXFP4_ERR_MISALIGNED

    def fwd(x=16, x_rows=8, ldx=24, row_index=None, offsets=64, rows=8, w=32, **change):
        return lib.mxfp4_grouped_forward(layer_struct(**change), x, x_rows, ldx, row_index, offsets, rows, w, None)

    def bwd(dy=16, lddy=8, offsets=64, rows=8, **change):
        return lib.mxfp4_grouped_backward(layer_struct(**change), dy, lddy, offsets, rows, None)

    assert lib.mxfp4_grouped_forward(None, 16, 8, 24, None, 64, 8, None, None) == bad
    assert fwd(offsets=None) == bad and fwd(x=None) == bad and fwd(rows=-1) == bad and fwd(rows=9) == bad
    assert fwd(groups=0) == bad and fwd(groups=2**40) == bad and fwd(N=2**31) == bad and fwd(y=None) == bad
    assert fwd(x_blobs=(None, 32, None, None)) == bad and fwd(x_blobs=(16, 32, 48, None)) == bad
    assert fwd(w_blobs=(None, 96, None, None), w=None) == bad
    assert fwd(ldx=28) == mis and fwd(w=40) == mis and fwd(x=20) == mis and fwd(y=0x1008) == mis
    assert fwd(K=20, ldx=24) == mis                  # W's rows of 20 elements are not 16 bytes apart
    assert lib.mxfp4_grouped_backward(None, 16, 8, 64, 8, None) == bad
    assert bwd(offsets=None) == bad and bwd(dy=None) == bad and bwd(lddy=7) == bad
    assert bwd(dx=None) == bad and bwd(dw=None) == bad
    for name in ("x_blobs", "w_blobs", "dy_blobs"):  # the col blobs of a training layer
        assert bwd(**{name: (16, 32, None, None)}) == bad
    assert bwd(dy=24) == mis and bwd(lddy=12) == mis and bwd(dw=0x3004) == mis


def test_layer_refusals():
    import torch
    from mxfp4_block_scaled_quantize_gb300.grouped import MXFP4GroupedLinear
    L = MXFP4GroupedLinear(2, 8, 24, 10, train=False, device="cpu")
    x, o = torch.zeros(4, 24, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    w = torch.zeros(2, 8, 24, dtype=torch.bfloat16)
    for args in ((x, None, o), (x, w.float(), o), (x, w[:, :, :16], o), (x.float(), w, o), (x[:, :16], w, o),
                 (x, w, o[:2]), (x, w, o.long()), (torch.zeros(11, 24, dtype=torch.bfloat16), w, o),
                 (x, w, o, torch.zeros(11, dtype=torch.int32)), (x, w, o, torch.zeros(4))):
        with pytest.raises(ValueError):
            L.forward(*args)
    with pytest.raises(ValueError):
        L.backward(x[:, :8].contiguous(), o)
    with pytest.raises(ValueError):
        MXFP4GroupedLinear(2, 8, 24, 10, device="cpu", out_dtype=torch.float16)


def test_no_usable_device_fails_loudly(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a CUDA device is present")
    gone = (abi.MXFP4_ERR_CUDA, abi.MXFP4_ERR_UNSUPPORTED_DEVICE)
    assert lib.mxfp4_quantize_grouped(0x10000, 8, 8, 8, None, 0x20000, 2, 8, 0x30000, 0x40000, None, None, None) in gone
    assert lib.mxfp4_gemm_grouped(0, 0x10000, 0x20000, 0x30000, 0x40000, 0x50000, 2, 8, 8, 24, 0x60000, 24, 0,
                                  None) in gone
    assert abi.status_string(abi.MXFP4_ERR_GROUPS).startswith("MXFP4_ERR_GROUPS")


def group_table(offsets, groups, rows):
    """csrc/group_table.cuh, chunk by chunk and lane by lane: starts, 128-row tiles before, refused."""
    start, tiles, bad = [0] * (groups + 1), [0] * (groups + 1), False
    top = total = 0
    for base in range(0, groups + 1, 32):
        cur = [offsets[min(base + lane, groups)] for lane in range(32)]
        last = offsets[min(base + 32, groups)]
        nxt = cur[1:] + [last]
        if any(c < top or c > rows or n < c or n > rows for c, n in zip(cur, nxt)):
            bad = True
            cur = [max(min(c, rows), top) for c in cur]
            nxt = [max(min(n, rows), top) for n in nxt]
            for lane in range(1, 32):
                cur[lane] = max(cur[lane], cur[lane - 1])
            nxt = [max(n, c) for n, c in zip(nxt, cur)]
            nxt = cur[1:] + [nxt[31]]
        for lane in range(32):
            e = base + lane
            if e <= groups:
                start[e], tiles[e] = cur[lane], total
            if e < groups:
                total += (nxt[lane] - cur[lane] + 127) // 128
        top = nxt[31]
    return start, tiles, bad


def test_group_table_stays_inside_the_buffers(lib):
    import random
    rng = random.Random(1)
    for _ in range(400):
        groups, rows = rng.choice([1, 2, 31, 32, 33, 64, 1024]), rng.choice([0, 1, 127, 128, 1000, 70000])
        o = [rng.randint(-2 * rows - 3, 3 * rows + 3) for _ in range(groups + 1)]
        if rng.random() < 0.5:
            o.sort()
        start, tiles, bad = group_table(o, groups, rows)
        assert all(0 <= s <= rows for s in start) and start == sorted(start)
        assert tiles == [sum((b - a + 127) // 128 for a, b in zip(start[:e], start[1:e + 1])) for e in range(groups + 1)]
        assert 128 * tiles[-1] <= abi.mxfp4_grouped_sizes(rows, 8, groups)[4]
        want, top = [], 0
        for x in o:
            top = max(top, min(max(x, 0), rows))
            want.append(top)
        assert start == want and bad == (want != o)



def test_waves_deal_every_tile_once(lib):
    # csrc/gemm_grouped.cu: cluster c takes tile w n + (c + w) % n of wave w
    for n in (1, 2, 5, 76):
        for total in (0, 1, n - 1, n, n + 1, 3 * n + 2, 500):
            got = []
            for c in range(n):
                w = 0
                while (i := w * n + (c + w) % n) < total:
                    got.append(i)
                    w += 1
            assert sorted(got) == list(range(total))
