"""medusa_linear_w4 where each case says which of its kernels it runs on: the forms of the kernel for many tokens, and sums that are
exact, or nearly, whatever the number of columns and of CTAs that share them.

The reference is worked out on the GPU in 64 bits by torch (and pinned to the numpy oracle here), as these layers are large."""
import ctypes

import numpy as np
import pytest

from oracle import verify as ov
from tests.helpers import to_dev
from tests.verify import U, bf16, dev_matrix, linear_bound, matrix

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

REGISTERS, EVEN, TILES = 0, 1, 2
OUT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def mg():
    import medusa_head_speculative_heads_gb300 as m
    m.build()
    return m


def division(mg, T, K, N):
    """(kernel, CTAs that share a tile, tokens and features of a tile, tiles, CTAs)"""
    d = (ctypes.c_int32 * 6)()
    assert mg.lib().medusa_linear_w4_test_division(T, K, N, d) == 0
    return list(d)


def reference(x, q, s, z):
    """(x W^T, sum of |x w|) in float64."""
    N, K = q.shape[0], q.shape[1] * 8
    place = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], device="cuda", dtype=torch.int32)
    e = ((q[:, :, None] >> place) & 15).view(N, K).float()
    each = K // s.shape[0]
    e -= 8 if z is None else (z & 127).float().t().repeat_interleave(each, 1)
    w = (s.float().t().repeat_interleave(each, 1) * e).bfloat16().double()  # 8 bits by 8: the product is exact in fp32
    return x.double() @ w.t(), x.double().abs() @ w.abs().t()


def layer(seed, T, K, N, G, zeros):
    rng = np.random.default_rng(seed)
    return to_dev(bf16(rng, T, K)), dev_matrix(matrix(rng, N, K, G, zeros))


def whole(seed, T, K, N, G, zeros):
    """Inputs -2 .. 2 and weights that are halves up to 30: a sum of 2^17 products and all its parts are exact in fp32."""
    assert K <= 1 << 17
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randint(-2, 3, (T, K), device="cuda", generator=g).bfloat16()
    q = torch.randint(-2 ** 31, 2 ** 31, (N, K // 8), device="cuda", generator=g).int()
    s = torch.exp2(torch.randint(-1, 2, (K // G, N), device="cuda", generator=g).float()).bfloat16()
    return x, (q, s, torch.randint(0, 16, (K // G, N), device="cuda", generator=g, dtype=torch.uint8) if zeros else None)


def check(got, x, m, out):
    y, size = reference(x, *m)
    off, most = (got.double() - y).abs().cpu().numpy(), linear_bound(y.cpu().numpy(), size.cpu().numpy(), x.shape[1], out)
    assert np.all(off <= most), float(np.max(off / most))


def test_the_reference_is_the_oracles(mg):
    rng = np.random.default_rng(3)
    for G, zeros in ((32, True), (64, False), (128, True)):
        x, m = bf16(rng, 5, 384), matrix(rng, 70, 384, G, zeros)
        if zeros:
            m[2][:] |= 128  # ignored
        want = ov.linear_w4(x, *m)
        for a, b in zip(reference(to_dev(x), *dev_matrix(m)), want):
            np.testing.assert_allclose(a.cpu().numpy(), b, rtol=0, atol=384 * 2.0 ** -53 * float(np.abs(want[1]).max()))


FORMS = [  # T, K, N, group, zeros, out.  Features that are not a multiple of 16: scales that are not loaded by TMA
    (700, 2048, 5000, 128, True, "bf16"),
    (700, 2048, 4992, 128, True, "f32"),
    (700, 2048, 5008, 128, False, "bf16"),
    (1500, 1120, 4001, 32, True, "bf16"),  # a block of columns that ends early
    (1500, 1120, 4016, 32, True, "f32"),
    (1500, 1120, 4016, 32, False, "bf16"),
    (3000, 544, 3501, 32, False, "f32"),
    (3000, 576, 3520, 64, True, "f32"),
    (3000, 576, 3519, 64, True, "bf16"),
    (200, 8192, 4001, 64, False, "bf16"),  # shared tiles
    (200, 8192, 4096, 128, True, "f32"),
    (171, 11008, 4096, 64, True, "bf16"),
    (171, 11008, 4095, 128, False, "f32"),
    (65, 65536, 256, 128, True, "bf16"),   # by eight CTAs
    (65, 65536, 250, 32, True, "f32"),
    (130, 65536, 64, 64, True, "bf16"),
    (129, 32768, 1100, 128, True, "f32"),
    (257, 16416, 900, 32, True, "bf16"),
    (257, 16448, 912, 64, True, "f32"),
]
IDS = ["-".join(map(str, s)) for s in FORMS]


@pytest.mark.parametrize("T,K,N,G,zeros,out", FORMS, ids=IDS)
def test_forms_for_many_tokens(mg, T, K, N, G, zeros, out):
    assert division(mg, T, K, N)[0] == TILES
    x, m = layer(T + K + N, T, K, N, G, zeros)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = mg.medusa_linear_w4(x, *m, out_dtype=OUT[out], d_status=st)
    assert mg.medusa_status_check(st) == 0
    check(got, x, m, out)


EXACT = [(TILES, *f) for f in FORMS] + [
    (REGISTERS, 1, 4096, 4096, 128, True, "f32"),
    (REGISTERS, 7, 5120, 13825, 32, True, "bf16"),
    (REGISTERS, 8, 8224, 1000, 32, False, "f32"),
    (REGISTERS, 16, 11008, 700, 64, True, "f32"),
    (EVEN, 1, 4096, 32000, 128, False, "f32"),
    (EVEN, 3, 65536, 16, 64, True, "f32"),
    (EVEN, 16, 16416, 1700, 32, True, "f32"),
    (EVEN, 25, 11008, 4096, 64, True, "bf16"),
    (EVEN, 64, 4096, 22016, 128, True, "f32"),
    (EVEN, 50, 16448, 999, 64, False, "f32"),
    (EVEN, 128, 4096, 4096, 128, True, "f32"),
    (EVEN, 171, 2048, 3001, 32, True, "bf16"),
]


@pytest.mark.parametrize("kernel,T,K,N,G,zeros,out", EXACT, ids=["-".join(map(str, s)) for s in EXACT])
def test_no_product_is_lost(mg, kernel, T, K, N, G, zeros, out):
    """Sums that are exact in any order: the result is right to the last bit."""
    assert division(mg, T, K, N)[0] == kernel
    x, m = whole(T + K + N, T, K, N, G, zeros)
    got = mg.medusa_linear_w4(x, *m, out_dtype=OUT[out])
    assert torch.equal(got, reference(x, *m)[0].float().to(OUT[out]))


def test_few_tokens_sums_are_not_cut_off(mg):
    """Up to 16 tokens of a layer on tensor memory have four sums a stream of blocks, two streams and up to eight CTAs.  Products up to
    255 x 127, all above zero, 512 of them in a sum at most: less than 2^24, so each sum is exact.  Eight sums a CTA and eight
    CTAs' are added with 7 and 7 roundings, so |error| <= 14 u y.  (With one sum a stream the tensor core would cut off bits: of
    2^26 it keeps multiples of 4.)"""
    N, G = 16, 128
    for T in (1, 7, 16):
        kernel, share = division(mg, T, 32768, N)[:2]
        assert kernel == EVEN and share == 8
        K = 8 * 8 * 512
        g = torch.Generator(device="cuda").manual_seed(T)
        x = (torch.randint(64, 128, (T, K), device="cuda", generator=g) * 2 + 1).bfloat16()
        q = torch.randint(-2 ** 31, 2 ** 31, (N, K // 8), device="cuda", generator=g).int()
        m = q, torch.full((K // G, N), -1.0, device="cuda", dtype=torch.bfloat16), torch.full((K // G, N), 127, device="cuda", dtype=torch.uint8)
        y = reference(x, *m)[0]
        assert y.min() > 2.0 ** 28
        assert ((mg.medusa_linear_w4(x, *m, out_dtype=torch.float32).double() - y).abs() <= 14 * U * y).all()


MANY = [(700, 2048, 5000, 64), (200, 8192, 4096, 128), (65, 65536, 250, 32)]


@pytest.mark.parametrize("T,K,N,G", MANY)
def test_rows_of_a_wider_buffer_and_outputs_given(mg, T, K, N, G):
    assert division(mg, T, K, N)[0] == TILES
    x, m = layer(T, T, K, N, G, True)
    wide = torch.full((T, K + 40), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :K] = x
    y = torch.full((T + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    got = mg.medusa_linear_w4(wide[:, :K], *m, y=y[1:T + 1])
    assert got.data_ptr() == y[1:].data_ptr() and (y[0] == 7).all() and (y[-1] == 7).all()
    check(got, x, m, "bf16")
    odd = torch.full((T * N + 1,), 7.0, device="cuda")[1:].view(T, N)  # 4-byte aligned only
    check(mg.medusa_linear_w4(x, *m, y=odd), x, m, "f32")
    scales = torch.empty(m[1].numel() + 1, dtype=torch.bfloat16, device="cuda")[1:].view(m[1].shape).copy_(m[1])  # 2-byte aligned only
    assert torch.equal(mg.medusa_linear_w4(x, m[0], scales, m[2]), got)


@pytest.mark.parametrize("T,K,N,G", MANY)
def test_what_is_not_a_number_stays_in_its_row_or_column(mg, T, K, N, G):
    assert division(mg, T, K, N)[0] == TILES
    x, (q, s, z) = layer(N, T, K, N, G, True)
    x[1, 100], x[T - 1, K - 1] = float("nan"), float("inf")
    s[2, 150], s[-1, 151], s[0, N - 1] = float("nan"), float("-inf"), -0.0
    got, want = mg.medusa_linear_w4(x, q, s, z, out_dtype=torch.float32).double(), reference(x, q, s, z)[0]
    assert torch.equal(got.isnan(), want.isnan())
    inf = want.isinf()
    assert torch.equal(got[inf], want[inf])
    fine = [t for t in range(T) if t not in (1, T - 1)], [n for n in range(N) if n not in (150, 151)]
    rows, cols = (torch.tensor(i, device="cuda") for i in fine)
    check(got[rows][:, cols], x[rows], (q[cols], s[:, cols], z[:, cols]), "f32")


@pytest.mark.parametrize("T,K,N,G", MANY)
def test_calls_repeat_bit_for_bit_eager_captured_and_at_once(mg, T, K, N, G):
    assert division(mg, T, K, N)[0] == TILES
    x, m = layer(K, T, K, N, G, True)
    first = mg.medusa_linear_w4(x, *m)
    check(first, x, m, "bf16")
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph):
        captured = mg.medusa_linear_w4(x, *m)
    outs = [torch.empty_like(first) for _ in range(2)]
    for _ in range(10):
        captured.zero_()
        graph.replay()
        mg.medusa_linear_w4(x, *m, y=outs[1], stream=side)
        mg.medusa_linear_w4(x, *m, y=outs[0])
        torch.cuda.synchronize()
        assert torch.equal(captured, first) and torch.equal(outs[0], first) and torch.equal(outs[1], first)
