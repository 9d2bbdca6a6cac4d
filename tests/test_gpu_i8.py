"""GPU parity of int8 row quantization and of the scaled int8 product.

Bounds, from the arithmetic of the calls: the quantization is exact (q and the scale are compared
bit for bit).  The product's sums are exact; float(sum), the two scalings and the bias round once
each (2^-24 relative), the store once more (half a step of the output type)."""
import numpy as np
import pytest
import torch

import block_quant_gemv_b200 as bqg
from oracle import i8 as oi
from tests.util import need_gpu

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.float16, torch.bfloat16]


def rows(seed, r, k, dtype, pitch=None):
    """Seeded rows on the device at a row pitch; what lies behind a row is poison."""
    g = torch.Generator().manual_seed(seed)
    x = torch.full((r, pitch or k), float("nan"), dtype=dtype)
    x[:, :k] = (torch.randn(r, k, generator=g) * torch.exp(torch.randn(r, 1, generator=g))).to(dtype)
    return x.cuda()[:, :k]


def int8_rows(seed, r, k, pitch=None):
    g = torch.Generator().manual_seed(seed)
    pitch = pitch or (k + 15) // 16 * 16
    q = torch.randint(-128, 128, (r, pitch), generator=g, dtype=torch.int8)
    return q.cuda()[:, :k]


def check_product(y, q, sx, w, sw, bias, where=""):
    ref = oi.product(q.cpu().numpy(), sx.cpu().numpy(), w.cpu().numpy(), sw.cpu().numpy(),
                     None if bias is None else bias.cpu().numpy())
    unbiased = ref if bias is None else ref - bias.cpu().numpy().astype(np.float64)
    half = torch.finfo(y.dtype).eps / 2
    bound = (3 * 2.0 ** -24 * np.abs(unbiased) + 2.0 ** -24 * np.abs(ref)) * (1 + 2 * half) + half * np.abs(ref)
    bound += torch.finfo(y.dtype).smallest_normal * half  # below the normal range steps stop shrinking
    got = y.detach().cpu().double().numpy()
    assert np.all(np.isfinite(got)), where
    worst = np.max(np.abs(got - ref) - bound)
    assert worst <= 0, f"{where}: {worst} above the bound"


# ---------------------------------------------------------------- quantization
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("r,k,pitch", [(1, 1, None), (3, 7, 11), (5, 32, None), (9, 1000, 1000), (17, 1023, 1030),
                                       (2, 1025, None), (3, 4096, 4104), (2, 8192, None), (2, 8209, 8211),
                                       (1, 40000, None), (300, 64, None)])
def test_quantize_bit_exact(r, k, pitch, dtype):
    need_gpu()
    X = rows(r * 1000 + k, r, k, dtype, pitch)
    q, s = bqg.quantize_rows_i8(X)
    ref_q, ref_s = oi.quantize_rows(X.float().cpu().numpy())
    assert q.dtype == torch.int8 and tuple(q.shape) == (r, k) and q.stride(0) % 16 == 0
    assert np.array_equal(s.cpu().numpy(), ref_s)
    assert np.array_equal(q.cpu().numpy(), ref_q)


def test_quantize_ties_go_to_even():
    """Rows of scale 1 and of scale 2^-3 holding every half: the quotient is an exact tie."""
    need_gpu()
    v = torch.arange(-253, 254, dtype=torch.float32) / 2
    v = torch.cat([v, torch.tensor([127.0])])
    X = torch.stack([v, v / 8, torch.nextafter(v, torch.full_like(v, 1e9)).clamp(max=127),
                     torch.nextafter(v, torch.full_like(v, -1e9)).clamp(min=-127)])
    X[2, -1] = X[3, -1] = 127.0
    q, s = bqg.quantize_rows_i8(X.cuda())
    ref_q, ref_s = oi.quantize_rows(X.numpy())
    assert np.array_equal(s.cpu().numpy(), ref_s) and ref_s[0] == 1 and ref_s[1] == 0.125
    assert np.array_equal(q.cpu().numpy(), ref_q)
    assert q[0].cpu().tolist()[:4] == [-126, -126, -126, -125]


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_odd_rows(dtype):
    """Rows of zeros, below the smallest scale, with Inf and with NaN; the largest finite value."""
    need_gpu()
    X = rows(3, 8, 2049, dtype)
    X[0] = 0
    X[1, 17], X[2, 2048], X[3, 0] = float("inf"), float("nan"), float("-inf")
    X[4] = 0
    X[4, 5] = torch.finfo(dtype).max
    X[5] *= 0
    X[5, 2047] = torch.finfo(dtype).smallest_normal
    q, s = bqg.quantize_rows_i8(X)
    ref_q, ref_s = oi.quantize_rows(X.float().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), ref_s, equal_nan=True)
    assert np.array_equal(q.cpu().numpy(), ref_q)
    assert torch.isnan(s[1:4]).all() and not q[1:4].any()


def test_quantize_leaves_the_rest_alone():
    """A caller's buffers: the bytes behind each row and the rows behind the last stay as they were."""
    need_gpu()
    X = rows(4, 5, 37, torch.bfloat16)
    buf = torch.full((8, 64), 77, dtype=torch.int8, device="cuda")
    s = torch.full((8,), 5.0, device="cuda")
    bqg.quantize_rows_i8(X, buf[:5, :37], s)
    assert (buf[:, 37:] == 77).all() and (buf[5:] == 77).all() and (s[5:] == 5).all()
    assert np.array_equal(buf[:5, :37].cpu().numpy(), oi.quantize_rows(X.float().cpu().numpy())[0])


# ---------------------------------------------------------------- product
SHAPES = [(1, 16, 1), (1, 2048, 256), (1, 4099, 77), (2, 33, 5), (3, 512, 130), (5, 1111, 9), (8, 640, 1001),
          (9, 64, 128), (9, 31, 3), (16, 128, 127), (17, 129, 129), (33, 1000, 200), (64, 256, 640), (100, 2051, 1000),
          (128, 4096, 512), (129, 300, 131), (200, 1024, 4096), (257, 96, 1), (300, 513, 2305), (1024, 640, 2176),
          (8, 65536, 20), (12, 65536, 140)]


@pytest.mark.parametrize("tokens,k,n", SHAPES)
@pytest.mark.parametrize("out", TYPES)
def test_product_matches_oracle(tokens, k, n, out):
    need_gpu()
    seed = tokens * 7919 + k * 31 + n
    q, w = int8_rows(seed, tokens, k), int8_rows(seed + 1, n, k)
    g = torch.Generator().manual_seed(seed)
    sx = (torch.rand(tokens, generator=g) * 1e-3 + 1e-4).cuda()
    sw = (torch.rand(n, generator=g) * 1e-2 + 1e-3).cuda()
    bias = torch.randn(n, generator=g).cuda() if (tokens + n) % 2 else None
    y = bqg.qgemm_i8(q, sx, w, sw, out_dtype=out, bias=bias)
    assert y.dtype == out and tuple(y.shape) == (tokens, n)
    check_product(y, q, sx, w, sw, bias, f"{tokens}x{k}x{n}")
    assert torch.equal(y, bqg.qgemm_i8(q, sx, w, sw, out_dtype=out, bias=bias))  # deterministic


def test_product_extreme_values():
    """Every value -128 at the largest k: the sums reach 2^30 exactly on both paths."""
    need_gpu()
    k = bqg.MAX_I8_COLS
    for tokens in (2, 20):
        q = torch.full((tokens, k), -128, dtype=torch.int8, device="cuda")
        w = torch.full((130, k), -128, dtype=torch.int8, device="cuda")
        y = bqg.qgemm_i8(q, torch.ones(tokens, device="cuda"), w, torch.ones(130, device="cuda"), torch.float32)
        assert (y == float(2 ** 30)).all()


def test_product_paths_agree_bit_for_bit():
    """The same token alone, among 8 (dp4a) and among many (tensor cores): the same bits."""
    need_gpu()
    q, w = int8_rows(1, 700, 1000), int8_rows(2, 333, 1000)
    sx, sw = torch.rand(700, device="cuda") + 0.5, torch.rand(333, device="cuda") + 0.5
    bias = torch.randn(333, device="cuda")
    y = bqg.qgemm_i8(q, sx, w, sw, torch.float32, bias)
    for a, b in ((0, 1), (3, 5), (10, 14), (20, 28), (30, 46), (64, 100), (100, 228), (100, 400)):
        assert torch.equal(bqg.qgemm_i8(q[a:b], sx[a:b], w, sw, torch.float32, bias), y[a:b]), (a, b)


@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("tokens,n,pitch", [(4, 65, 70), (30, 65, 71), (30, 64, 64), (300, 131, 137), (300, 130, 140)])
def test_product_into_strided_rows(tokens, n, pitch, out):
    """Y inside a larger buffer at odd and even pitches and offsets: nothing else is written."""
    need_gpu()
    k = 200
    q, w = int8_rows(3, tokens, k, 256), int8_rows(4, n, k, 224)
    sx, sw = torch.rand(tokens, device="cuda"), torch.rand(n, device="cuda")
    for first in (0, 1):
        buf = torch.full((tokens + 3, pitch + 1), -7.0, dtype=out, device="cuda")
        view = buf[1:1 + tokens, first:first + n]
        bqg.qgemm_i8(q, sx * 1e-3, w, sw, Y=view)
        check_product(view, q, sx * 1e-3, w, sw, None)
        rest = buf.clone()
        rest[1:1 + tokens, first:first + n] = -7.0
        assert (rest == -7.0).all()


def test_product_nonfinite_row_stays_in_its_row():
    need_gpu()
    for tokens in (6, 40):
        X = rows(5, tokens, 96, torch.float16)
        X[2, 50] = float("inf")
        q, s = bqg.quantize_rows_i8(X)
        w, sw = int8_rows(6, 70, 96), torch.rand(70, device="cuda") * 1e-2
        y = bqg.qgemm_i8(q, s, w, sw, torch.float32)
        assert torch.isnan(y[2]).all()
        keep = [t for t in range(tokens) if t != 2]
        check_product(y[keep], q[keep], s[keep], w, sw, None)


@pytest.mark.parametrize("tokens", [5, 12])
def test_product_offsets_past_32_bits(tokens):
    """Row pitches that put the last rows of X, W and Y beyond 4 GB."""
    need_gpu()
    k, n, pitch = 48, 12, 1 << 29
    q, w = int8_rows(7, tokens, k), int8_rows(8, n, k)
    bx = torch.empty(pitch * (tokens - 1) + 64, dtype=torch.int8, device="cuda")
    bw = torch.empty(pitch * (n - 1) + 64, dtype=torch.int8, device="cuda")
    by = torch.empty((pitch // 2) * (tokens - 1) + n, dtype=torch.float32, device="cuda")
    X, W = bx.as_strided((tokens, k), (pitch, 1)), bw.as_strided((n, k), (pitch, 1))
    Y = by.as_strided((tokens, n), (pitch // 2, 1))
    X.copy_(q)
    W.copy_(w)
    sx, sw = torch.rand(tokens, device="cuda"), torch.rand(n, device="cuda")
    bqg.qgemm_i8(X, sx, W, sw, Y=Y)
    check_product(Y, q, sx, w, sw, None)


# ---------------------------------------------------------------- streams, graphs, a run of both
def test_quantize_and_product_in_a_graph_and_on_a_stream():
    need_gpu()
    X = rows(9, 48, 1024, torch.bfloat16)
    w, sw = bqg.quantize_rows_i8(rows(10, 500, 1024, torch.float32))  # the weights, quantized once
    Y = torch.zeros(48, 500, dtype=torch.bfloat16, device="cuda")
    Xq = torch.empty(48, 1024, dtype=torch.int8, device="cuda")
    s = torch.empty(48, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step():
        bqg.quantize_rows_i8(X, Xq, s)
        bqg.qgemm_i8(Xq, s, w, sw, Y=Y)
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    check_product(Y, Xq, s, w, sw, None, "side stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            step()
    for seed in (11, 12):
        X.copy_(rows(seed, 48, 1024, torch.bfloat16))
        Y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        ref_q, ref_s = oi.quantize_rows(X.float().cpu().numpy())
        assert np.array_equal(Xq.cpu().numpy(), ref_q) and np.array_equal(s.cpu().numpy(), ref_s)
        check_product(Y, Xq, s, w, sw, None, "graph replay")


def test_two_streams_at_once():
    need_gpu()
    w, sw = int8_rows(20, 900, 768), torch.rand(900, device="cuda") * 1e-3
    jobs = []
    for i in range(4):
        q, sx = int8_rows(21 + i, 40 + i, 768), torch.rand(40 + i, device="cuda")
        jobs.append((q, sx, torch.empty(40 + i, 900, device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for q, sx, Y, st in jobs:
            with torch.cuda.stream(st):
                bqg.qgemm_i8(q, sx, w, sw, Y=Y)
    torch.cuda.synchronize()
    for q, sx, Y, _ in jobs:
        check_product(Y, q, sx, w, sw, None)


# ---------------------------------------------------------------- refusals that need device tensors
def test_binding_refusals():
    need_gpu()
    q = torch.zeros(4, 32, dtype=torch.int8, device="cuda")
    one = torch.ones(4, device="cuda")
    with pytest.raises(TypeError):
        bqg.quantize_rows_i8(q)                                    # int8 input
    with pytest.raises(ValueError):
        bqg.quantize_rows_i8(torch.ones(8, device="cuda"))          # not 2-D
    with pytest.raises(ValueError):
        bqg.quantize_rows_i8(torch.ones(8, 3, device="cuda").t())  # columns not contiguous
    with pytest.raises(ValueError):
        bqg.quantize_rows_i8(torch.ones(4, 16, device="cuda"), q)   # Xq of another width
    with pytest.raises(bqg.BQGError):
        bqg.quantize_rows_i8(torch.ones(4, 33, device="cuda"), torch.zeros(4, 33, dtype=torch.int8, device="cuda"))
    with pytest.raises(TypeError):
        bqg.qgemm_i8(q, one, q, one, out_dtype=torch.int32)
    with pytest.raises(ValueError):
        bqg.qgemm_i8(q, one, q[:, :16], one)                        # another k
    with pytest.raises(ValueError):
        bqg.qgemm_i8(q, one[:3], q, one)                            # too few scales
    with pytest.raises(ValueError):
        bqg.qgemm_i8(q, one, q, one, bias=one[:2])
    with pytest.raises(ValueError):
        bqg.qgemm_i8(q, one, q, one, Y=torch.empty(4, 5, device="cuda"))
    with pytest.raises(ValueError):
        bqg.qgemm_i8(q, one, q, one[:0])
    odd = torch.zeros(4, 40, dtype=torch.int8, device="cuda")[:, :33]
    with pytest.raises(bqg.BQGError):                               # a pitch that is no multiple of 16
        bqg.qgemm_i8(odd, one, odd, one)
    with pytest.raises(bqg.BQGError):                               # rows that start off a 16-byte boundary
        flat = torch.zeros(4 * 48 + 8, dtype=torch.int8, device="cuda")
        bqg.qgemm_i8(flat[8:].view(4, 48)[:, :32], one, q, one)
    with pytest.raises(ValueError):                                 # rows on top of one another
        bqg.qgemm_i8(q, one, q, one, Y=torch.empty(4, device="cuda").expand(4, 4))
