"""E4M3 products with block scales against 64-bit definitions.

Rounding: bytes and scales are those of the definition, exactly.  Products:
a block's 128 products are exact and summed in float32 by the tensor cores,
the blocks' scaled sums in float32, so with B blocks, up to 8 CTAs a tile and
every addition off by at most a last place (2^-23 relative; the tensor cores
may cut where others round) of a sum no larger than the magnitudes' sum R, and
3 roundings in a factor and its product: (128 + B + 8 + 3) 2^-23 R, and one
rounding to the result's type.
"""
import numpy as np
import pytest
import torch

import step_ref as ref

pytestmark = pytest.mark.gpu

BF16, FP16, F32 = torch.bfloat16, torch.float16, torch.float32


def _activations(n, cols, kind, seed, spread=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((n, cols), generator=g, device="cuda")
    if spread:  # magnitudes from subnormal results to saturating ones
        x *= torch.exp2(torch.randint(-12, 12, (n, cols), generator=g, device="cuda").float())
    return x.to(kind)


def _quantized(afx, x, pad=0, scale_pad=0):
    n, cols = x.shape
    width = -(-cols // 16) * 16 + pad
    q = torch.full((n, width), 0xAB, dtype=torch.uint8, device="cuda")
    scales = torch.full((-(-cols // 128), n + scale_pad), -7.0, device="cuda")
    afx.afx_fp8_quantize(x, q, scales[:, :n])
    assert (q[:, cols:] == 0xAB).all() and (scales[:, n:] == -7).all()
    return q, scales[:, :n]


def _check_quantized(x, q, scales):
    values, want = ref.quantize(x.float().cpu().numpy())
    assert np.array_equal(scales.cpu().numpy(), want, equal_nan=True)
    got = ref.e4m3_values()[q[:, :x.shape[1]].cpu().numpy()]
    assert np.array_equal(got, values, equal_nan=True)


@pytest.mark.parametrize("kind", [BF16, FP16, F32])
@pytest.mark.parametrize("n,cols", [(1, 1), (1, 128), (3, 127), (7, 129), (8, 512), (9, 1000), (65, 384), (130, 5120), (1, 20_001)])
def test_rounding(afx, kind, n, cols):
    x = _activations(n, cols, kind, n * 1000 + cols)
    _check_quantized(x, *_quantized(afx, x))


def test_rounding_ties_and_ends(afx):
    # every E4M3 value, every point half way between two, their neighbours; a scale of 1
    v = torch.tensor(ref.e4m3_values()[:127])
    v = torch.cat([v, (v[1:] + v[:-1]) / 2, torch.tensor([448.0])]).float()
    v = torch.cat([v, torch.nextafter(v, torch.full_like(v, 1e9)).clamp(max=448), torch.nextafter(v, torch.zeros_like(v))])
    v = torch.cat([v, -v])
    rows = torch.zeros((-(-len(v) // 127), 128))
    for i in range(rows.shape[0]):
        part = v[i * 127:(i + 1) * 127]
        rows[i, :len(part)] = part
        rows[i, 127] = 448.0
    x = rows.cuda()
    q, scales = _quantized(afx, x)
    assert (scales == 1).all()
    _check_quantized(x, q, scales)


def test_rounding_of_zeros_tiny_and_special_values(afx):
    x = torch.zeros((6, 300), device="cuda")
    x[1] = 1e-42
    x[2, 5] = float("inf")
    x[3, 130] = float("nan")
    x[4] = 3e38
    x[5] = -2.0 ** -126
    q, scales = _quantized(afx, x)
    _check_quantized(x, q, scales)
    assert (q[0, :300] == 0).all() and (scales[:, 0] == 2.0 ** -126).all()
    assert scales[0, 2].isnan() and scales[1, 3].isnan() and (q[2, :128] & 127 == 127).all() and scales[0, 3] == 2.0 ** -126


def test_rounding_of_strided_rows(afx):
    wide = _activations(33, 1001, BF16, 5)
    for x in (wide[:, 1:900], wide[::2, 3:515], wide[:, 8:136]):
        _check_quantized(x, *_quantized(afx, x, pad=16, scale_pad=3))
    # bytes that start anywhere
    x = wide[:, :260].contiguous()
    q = torch.zeros(33 * 263 + 1, dtype=torch.uint8, device="cuda")[1:].view(33, 263)
    scales = torch.zeros((3, 33), device="cuda")
    afx.afx_fp8_quantize(x, q, scales)
    _check_quantized(x, q, scales)


def _weights(rows, cols, seed, width=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.randint(0, 256, (rows, width or cols), generator=g, device="cuda").to(torch.uint8)
    w[w & 127 == 127] = 0  # no NaN
    scales = torch.rand((-(-rows // 128), -(-cols // 128)), generator=g, device="cuda") * 1e-3 + 1e-5
    return w[:, :cols], scales


def _values(q, cols):
    return torch.tensor(ref.e4m3_values(), device="cuda")[q[:, :cols].long()]


def _check_product(w, w_scales, q, x_scales, y):
    cols = w.shape[1]
    want, reach = ref.product(_values(w, cols), w_scales, _values(q, cols), x_scales)
    bound = (128 + x_scales.shape[0] + 8 + 3) * 2.0 ** -23 * reach
    bound = bound + ref.round_error(want.abs() + bound, y.dtype)
    worst = ((y.double() - want).abs() / bound).max().item()
    assert worst <= 1, worst


def _product(afx, w, w_scales, q, x_scales, kind, status=None):
    y = torch.full((q.shape[0], w.shape[0]), 77.0, dtype=kind, device="cuda")
    afx.afx_fp8_product(w, w_scales, q, x_scales, y, status_dev=status)
    return y


# token counts around a tile's and its eighths, row counts around the blocks', few and many steps
SHAPES = [(1, 1, 16), (1, 128, 128), (2, 100, 144), (7, 129, 256), (8, 255, 1024), (16, 300, 8192), (31, 1024, 5120), (33, 64, 400),
          (64, 640, 2048), (65, 1000, 1040), (127, 256, 128), (128, 512, 640), (129, 384, 272), (200, 7, 4096), (257, 1100, 1008),
          (500, 3000, 512), (1, 20_000, 256), (3, 128, 40_000)]


@pytest.mark.parametrize("kind", [BF16, FP16, F32])
@pytest.mark.parametrize("n,rows,cols", SHAPES)
def test_product(afx, kind, n, rows, cols):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = _activations(n, cols, BF16, n + rows, spread=False)
    q, x_scales = _quantized(afx, x)
    w, w_scales = _weights(rows, cols, cols)
    if kind == FP16:
        w_scales = w_scales / 64  # sums stay below 65504
    y = _product(afx, w, w_scales, q, x_scales, kind, status)
    _check_product(w, w_scales, q, x_scales, y)
    assert status.item() == 0
    assert torch.equal(y, _product(afx, w, w_scales, q, x_scales, kind))  # the same bits again


@pytest.mark.parametrize("n", [5, 300])
def test_product_of_odd_columns_and_strided_rows(afx, n):
    # columns that end inside 16 bytes; what lies behind them is NaN
    for cols in (1, 15, 127, 129, 333):
        width = -(-cols // 16) * 16 + 32
        w, w_scales = _weights(200, cols, 3, width=width)
        torch.as_strided(w, (200, width - cols), (width, 1), cols).fill_(0x7F)
        x = _activations(n, cols, F32, 4, spread=False)
        q, x_scales = _quantized(afx, x, pad=16, scale_pad=5)
        q[:, cols:] = 0x7F
        _check_product(w, w_scales, q, x_scales, _product(afx, w, w_scales, q, x_scales, F32))


def test_product_into_strided_rows(afx):
    for n, rows, offset, width in ((40, 96, 3, 103), (300, 64, 32, 128), (300, 160, 1, 161), (140, 70, 8, 80)):
        x = _activations(n, 256, F32, 9, spread=False)
        q, x_scales = _quantized(afx, x)
        w, w_scales = _weights(rows, 256, 8)
        for kind in (BF16, F32):
            whole = torch.full((n + 1, width), 5.0, dtype=kind, device="cuda")
            y = whole[:n, offset:offset + rows]
            afx.afx_fp8_product(w, w_scales, q, x_scales, y)
            _check_product(w, w_scales, q, x_scales, y)
            assert (whole[n] == 5).all() and (whole[:, :offset] == 5).all() and (whole[:, offset + rows:] == 5).all()


def test_product_of_special_values(afx):
    x = _activations(140, 300, F32, 1, spread=False)
    x[3, 7] = float("nan")
    x[130] = 0
    q, x_scales = _quantized(afx, x)
    w, w_scales = _weights(260, 300, 2, width=304)
    w[200, 299] = 0x7F
    w_scales[1, 1] = float("inf")
    y = _product(afx, w, w_scales, q, x_scales, F32)
    assert y[3].isnan().all() and y[:, 200].isnan().all()
    others = [t for t in range(140) if t not in (3, 130)]
    assert y[others][:, :128].isfinite().all() and y[others][:, 256:].isfinite().all()
    assert not y[others][:, 128:256].isfinite().any()
    assert (y[130, :128] == 0).all()


def test_product_largest_and_smallest_scales(afx):
    # each step's factor is far from the sums': no step's may be lost
    q = torch.full((2, 256), 0x38, dtype=torch.uint8, device="cuda")  # 1.0
    w = torch.full((128, 256), 0x38, dtype=torch.uint8, device="cuda")
    x_scales = torch.tensor([[2.0 ** 60, 2.0 ** -60], [2.0 ** -60, 2.0 ** 60]], device="cuda")
    w_scales = torch.tensor([[2.0 ** -60, 2.0 ** 60]], device="cuda")
    y = _product(afx, w, w_scales, q, x_scales, F32)
    assert (y[0] == 256).all() and (y[1] == 128 * 2.0 ** 120).all()


def test_restored_weights(afx):
    """Weights out of a container, restored and multiplied on one stream."""
    from weight_streaming_canonical_gb300 import synth
    rows, cols = 384, 512
    bits = synth.normal_e4m3(rows * cols, seed=3)
    container, desc = afx.encode(bits, fmt=afx.AFX_FMT_E4M3)
    w = torch.empty((rows, cols), dtype=torch.uint8, device="cuda")
    x = _activations(19, cols, BF16, 6, spread=False)
    w_scales = torch.rand((3, 4), device="cuda") + 0.5
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.zeros((19, cols), dtype=torch.uint8, device="cuda")
    x_scales = torch.zeros((4, 19), device="cuda")
    y = torch.zeros((19, rows), device="cuda")
    afx.afx_decode(desc, torch.from_numpy(container).cuda(), w.view(-1), status_dev=status)
    afx.afx_fp8_quantize(x, q, x_scales)
    afx.afx_fp8_product(w, w_scales, q, x_scales, y, status_dev=status)
    assert np.array_equal(w.cpu().numpy().reshape(-1), bits) and status.item() == 0
    _check_product(w, w_scales, q, x_scales, y)


def test_captured_and_on_two_streams(afx):
    x = [_activations(n, 1024, BF16, n, spread=False) for n in (6, 6)]
    w, w_scales = _weights(512, 1024, 5)
    sets = [(torch.zeros((6, 1024), dtype=torch.uint8, device="cuda"), torch.zeros((8, 6), device="cuda"), torch.zeros((6, 512), device="cuda"))
            for _ in range(2)]

    def both(i, stream):
        q, s, y = sets[i]
        afx.afx_fp8_quantize(x[i], q, s, stream=stream)
        afx.afx_fp8_product(w, w_scales, q, s, y, stream=stream)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(0, torch.cuda.current_stream())
    other = torch.cuda.Stream()
    for turn in range(3):
        x[0].copy_(_activations(6, 1024, BF16, 100 + turn, spread=False))
        other.wait_stream(torch.cuda.current_stream())
        both(1, other)
        graph.replay()
        torch.cuda.current_stream().wait_stream(other)
        for q, s, y in sets:
            _check_product(w, w_scales, q, s, y)


def test_nothing_to_do(afx):
    e = torch.empty
    afx.afx_fp8_quantize(e((0, 64), device="cuda"), e((0, 64), dtype=torch.uint8, device="cuda"), e((1, 0), device="cuda"))
    w, w_scales = _weights(128, 64, 1)
    afx.afx_fp8_product(w, w_scales, e((0, 64), dtype=torch.uint8, device="cuda"), e((1, 0), device="cuda"), e((0, 128), device="cuda"))


def test_rounding_at_borders_of_scales(afx):
    """Quotients beside the borders between two E4M3 values, for scales from the smallest to the largest and any last bits."""
    g = torch.Generator().manual_seed(77)
    rows = 4000
    scale = torch.exp2(torch.randint(-126, 118, (rows,), generator=g).float()) * (1 + torch.rand(rows, generator=g))
    top = (scale.double() * 448).clamp(max=3.3e38).float()
    v = torch.tensor(ref.e4m3_values()[:127])
    border = ((v[1:] + v[:-1]) / 2)[torch.randint(0, 126, (rows, 127), generator=g)]
    x = (border * scale.double()[:, None]).float()
    bits = x.view(torch.int32) + torch.randint(-2, 3, x.shape, generator=g).to(torch.int32)
    x = torch.minimum(bits.clamp(min=0).view(torch.float32), top[:, None])
    x = torch.cat([x, top[:, None]], 1).cuda()
    q, scales = _quantized(afx, x)
    _check_quantized(x, q, scales)


# shapes whose tiles go to pairs of CTAs: 192 and 256 rows a tile; last tiles of a few tokens or rows, columns that end inside a
# block, one block, several tiles a pair, long sums
PAIRS = [(501, 7168, 384), (512, 7296, 1000), (700, 5120, 640), (2000, 9999, 384), (777, 14_000, 1000), (3000, 5000, 128), (700, 5120, 17_408)]


@pytest.mark.parametrize("n,rows,cols", PAIRS)
def test_product_by_pairs(afx, n, rows, cols):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = _activations(n, cols, BF16, n + rows, spread=False)
    q, x_scales = _quantized(afx, x)
    w, w_scales = _weights(rows, cols, cols, width=-(-cols // 16) * 16)
    for kind in (BF16, F32):
        whole = torch.full((n + 1, rows + 5), 5.0, dtype=kind, device="cuda")
        for y in (torch.full((n, rows), 77.0, dtype=kind, device="cuda"), whole[:n, 1:rows + 1]):
            afx.afx_fp8_product(w, w_scales, q, x_scales, y, status_dev=status)
            _check_product(w, w_scales, q, x_scales, y)
        assert (whole[n] == 5).all() and (whole[:, 0] == 5).all() and (whole[:, rows + 1:] == 5).all()
        assert torch.equal(y, _product(afx, w, w_scales, q, x_scales, kind))
    assert status.item() == 0


def test_pairs_with_special_values(afx):
    x = _activations(700, 384, F32, 1, spread=False)
    x[300, 7] = float("nan")
    x[650] = 0
    q, x_scales = _quantized(afx, x)
    w, w_scales = _weights(5120, 384, 2)
    w[3000, 383] = 0x7F
    w_scales[2, 1] = float("inf")
    y = _product(afx, w, w_scales, q, x_scales, F32)
    assert y[300].isnan().all() and y[:, 3000].isnan().all()
    rest = torch.ones_like(y, dtype=torch.bool)
    rest[300] = rest[:, 3000] = rest[:, 256:384] = False
    assert y[rest].isfinite().all() and not y[:300, 256:384].isfinite().any()
    assert (y[650, :256] == 0).all()


def test_products_side_by_side(afx):
    """Calls on two streams at once, of every shape of tile, have their own results."""
    sets = []
    for i, (n, rows, cols) in enumerate([(700, 5120, 640), (501, 7168, 384), (64, 640, 2048), (300, 20_000, 256), (5, 1024, 5120)]):
        q, x_scales = _quantized(afx, _activations(n, cols, BF16, i, spread=False))
        sets.append((*_weights(rows, cols, i), q, x_scales))
    want = [_product(afx, *s, F32) for s in sets]
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[torch.empty_like(w) for w in want] for _ in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for k, stream in enumerate(streams):
            for i in range(len(sets)):
                at = (i + 2 * k) % len(sets)
                afx.afx_fp8_product(*sets[at], got[k][at], stream=stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for one in got for a, b in zip(one, want))
