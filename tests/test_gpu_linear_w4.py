"""medusa_linear_w4 and medusa_w4_quantize against the float64 oracle (bounds: tests/verify.py)."""
import numpy as np
import pytest

import workloads as wl
from oracle import verify as ov
from tests.helpers import to_dev, to_host
from tests.verify import bf16, check_linear, dev_matrix, dev_words, host_words, matrix, value

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mg():
    import medusa_head_speculative_heads_gb300 as m
    m.build()
    return m


SHAPES = [  # T, K, N, group, zeros, out
    (1, 32, 1, 32, True, "bf16"),       # the least there is
    (1, 4096, 512, 128, True, "bf16"),
    (1, 4096, 777, 128, False, "f32"),  # odd rows, symmetric
    (1, 1152, 16, 64, True, "f32"),     # 9 blocks of columns
    (2, 96, 17, 32, True, "bf16"),      # a block of columns that ends early
    (3, 160, 130, 32, False, "f32"),
    (7, 5120, 129, 32, True, "bf16"),
    (8, 512, 128, 64, True, "f32"),
    (9, 512, 127, 64, True, "f32"),     # one token more than a tile
    (16, 640, 48, 128, True, "bf16"),
    (17, 640, 256, 64, False, "bf16"),
    (31, 1024, 300, 128, True, "f32"),
    (33, 1024, 300, 32, True, "bf16"),
    (64, 4096, 640, 128, True, "bf16"),
    (64, 96, 5, 32, True, "f32"),
    (65, 2048, 1, 64, True, "bf16"),
    (100, 11008, 256, 64, True, "f32"),
    (128, 128, 4000, 128, False, "bf16"),
    (171, 1376, 513, 32, True, "bf16"),
    (256, 256, 129, 128, True, "f32"),
    (257, 384, 1000, 128, True, "bf16"),
    (700, 2048, 383, 64, True, "bf16"),
    (2050, 64, 130, 64, False, "f32"),
]


@pytest.mark.parametrize("T,K,N,G,zeros,out", SHAPES, ids=["-".join(map(str, s)) for s in SHAPES])
def test_parity(mg, T, K, N, G, zeros, out):
    rng = np.random.default_rng(T * 31 + K + N)
    x, m = bf16(rng, T, K), matrix(rng, N, K, G, zeros)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = mg.medusa_linear_w4(to_dev(x), *dev_matrix(m), out_dtype=torch.float32 if out == "f32" else torch.bfloat16, d_status=st)
    assert mg.medusa_status_check(st) == 0
    check_linear(got, x, m, out)


SMALL_LAYERS = [  # of more than 64 tokens, in several tiles of tokens
    (65, 64, 20, 64, True, "bf16"),
    (70, 2080, 1000, 32, True, "f32"),
    (128, 2048, 2048, 128, True, "bf16"),
    (129, 1536, 2049, 64, False, "f32"),
    (256, 4096, 4096, 128, True, "bf16"),
    (333, 512, 3000, 64, True, "bf16"),
    (1000, 2048, 512, 128, False, "f32"),
    (2300, 256, 640, 32, True, "bf16"),
]


@pytest.mark.parametrize("T,K,N,G,zeros,out", SMALL_LAYERS, ids=["-".join(map(str, s)) for s in SMALL_LAYERS])
def test_parity_of_small_layers(mg, T, K, N, G, zeros, out):
    test_parity(mg, T, K, N, G, zeros, out)


FEW_TOKENS = [  # layers that are large for their few tokens, and those just below
    (1, 2304, 16384, 128, True, "bf16"),
    (1, 2016, 16385, 32, False, "f32"),
    (3, 8224, 5000, 32, True, "bf16"),
    (8, 8192, 4865, 64, True, "f32"),
    (8, 4096, 9729, 128, False, "bf16"),
    (9, 4128, 4100, 32, True, "f32"),
    (12, 1600, 10500, 64, True, "bf16"),
    (16, 4096, 4097, 128, False, "f32"),
    (16, 1024, 9728, 64, True, "bf16"),
    (16, 128, 32768, 128, True, "bf16"),
]


@pytest.mark.parametrize("T,K,N,G,zeros,out", FEW_TOKENS, ids=["-".join(map(str, s)) for s in FEW_TOKENS])
def test_parity_of_few_tokens(mg, T, K, N, G, zeros, out):
    test_parity(mg, T, K, N, G, zeros, out)


MORE_SHAPES = [  # many tiles of few blocks, tiles shared by two to eight CTAs, parts of one block
    (64, 128, 40000, 128, True, "bf16"),
    (20, 256, 30000, 64, False, "f32"),
    (64, 384, 20000, 128, True, "bf16"),
    (33, 32, 1024, 32, True, "f32"),
    (64, 1152, 22016, 128, True, "bf16"),
    (48, 1408, 2064, 128, True, "f32"),
    (17, 2048, 100, 64, True, "bf16"),
    (64, 4096, 4096, 32, False, "bf16"),
    (24, 640, 8193, 128, True, "bf16"),
    (3, 640, 9, 128, True, "f32"),
    (100, 256, 30000, 64, True, "bf16"),
    (520, 384, 5000, 128, False, "bf16"),
]


@pytest.mark.parametrize("T,K,N,G,zeros,out", MORE_SHAPES, ids=["-".join(map(str, s)) for s in MORE_SHAPES])
def test_parity_of_the_work_divided_otherwise(mg, T, K, N, G, zeros, out):
    test_parity(mg, T, K, N, G, zeros, out)


@pytest.mark.parametrize("T", [1, 5, 12, 30, 64, 300])
def test_every_element_and_place_of_a_word(mg, T):
    """Whole-numbered weights and inputs: the result is exact, whatever was mixed up."""
    rng = np.random.default_rng(T)
    K, N = 256, 144
    q = rng.integers(0, 16, (N, K))
    s = wl.to_bf16_bits(np.ldexp(1.0, rng.integers(-2, 3, (K // 32, N))).astype(np.float32))
    z = rng.integers(0, 128, (K // 32, N)).astype(np.uint8)
    x = wl.to_bf16_bits(rng.integers(-4, 5, (T, K)).astype(np.float32))
    want, _ = ov.linear_w4(x, ov.pack(q), s, z)
    got = mg.medusa_linear_w4(to_dev(x), dev_words(ov.pack(q)), to_dev(s), to_dev(z), out_dtype=torch.float32)
    np.testing.assert_array_equal(value(got), want)
    z |= 128  # the top bit is ignored
    again = mg.medusa_linear_w4(to_dev(x), dev_words(ov.pack(q)), to_dev(s), to_dev(z), out_dtype=torch.float32)
    assert torch.equal(got, again)


@pytest.mark.parametrize("T", [1, 20, 130])
def test_rows_of_a_wider_buffer_and_outputs_given(mg, T):
    rng = np.random.default_rng(T)
    K, N, gap = 384, 70, 40
    wide, m = bf16(rng, T, K + gap), matrix(rng, N, K, 128)
    wide[:, K:] = 0x7FC0  # NaN behind the rows
    x = to_dev(wide)[:, :K]
    y = torch.full((T + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    got = mg.medusa_linear_w4(x, *dev_matrix(m), y=y[1:T + 1])
    assert got.data_ptr() == y[1:].data_ptr() and (y[0] == 7).all() and (y[-1] == 7).all()
    check_linear(got, wide[:, :K], m, "bf16")
    odd = torch.full((T * N + 1,), 7.0, device="cuda")[1:].view(T, N)  # 4-byte aligned only
    check_linear(mg.medusa_linear_w4(x, *dev_matrix(m), y=odd), wide[:, :K], m, "f32")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = mg.medusa_linear_w4(x, *dev_matrix(m), stream=s)
    s.synchronize()
    assert torch.equal(other, got)


@pytest.mark.parametrize("T", [3, 40, 200])
def test_what_is_not_a_number_stays_in_its_row_or_column(mg, T):
    rng = np.random.default_rng(T)
    K, N = 512, 200
    x, (w, s, z) = bf16(rng, T, K), matrix(rng, N, K, 64)
    x[1, 100], x[2, 5] = 0x7FC0, 0x7F80          # NaN, +inf
    s[2, 150], s[3, 151], s[0, 152] = 0x7FC0, 0xFF80, 0x8000  # NaN, -inf, -0
    want, _ = ov.linear_w4(x, w, s, z)
    got = value(mg.medusa_linear_w4(to_dev(x), dev_words(w), to_dev(s), to_dev(z), out_dtype=torch.float32))
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    inf = np.isinf(want)
    np.testing.assert_array_equal(got[inf], want[inf])
    ok = np.isfinite(want)
    assert ok.sum() >= (T - 2) * (N - 2) and np.allclose(got[ok], want[ok], rtol=1e-4, atol=1e-4)


@pytest.mark.parametrize("T,K,N", [(1, 4096, 4096), (8, 2048, 1000), (24, 4096, 512), (64, 4096, 4096), (300, 1024, 999)])
def test_calls_repeat_bit_for_bit_eager_captured_and_at_once(mg, T, K, N):
    rng = np.random.default_rng(N)
    x, m = to_dev(bf16(rng, T, K)), dev_matrix(matrix(rng, N, K, 128))
    first = mg.medusa_linear_w4(x, *m)
    assert torch.isfinite(first.float()).all()
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


def test_no_rows(mg):
    rng = np.random.default_rng(0)
    y = mg.medusa_linear_w4(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), *dev_matrix(matrix(rng, 5, 64, 32)))
    assert y.shape == (0, 5)


def test_the_same_as_the_bf16_layer_on_the_weights_it_stands_for(mg):
    rng = np.random.default_rng(9)
    x, m = bf16(rng, 64, 1024), matrix(rng, 384, 1024, 64)
    w = ov.bf16_bits(ov.weights(*m))
    a, b = mg.medusa_linear_w4(to_dev(x), *dev_matrix(m)), mg.medusa_linear(to_dev(x), to_dev(w))
    assert torch.allclose(a.float(), b.float(), rtol=2.0 ** -7, atol=1e-3)


def test_refusals(mg):
    rng = np.random.default_rng(0)
    x, (q, s, z) = to_dev(bf16(rng, 4, 128)), dev_matrix(matrix(rng, 6, 128, 64))
    with pytest.raises(ValueError, match="groups"):
        mg.medusa_linear_w4(x, q, s[:1].expand(3, 6), z)
    with pytest.raises(ValueError, match="qweight"):
        mg.medusa_linear_w4(x, q[:, :8], s, z)
    with pytest.raises(ValueError, match="zeros"):
        mg.medusa_linear_w4(x, q, s, z[:, :5])
    with pytest.raises(ValueError, match="scales"):
        mg.medusa_linear_w4(x, q, s.float(), z)
    with pytest.raises(TypeError):
        mg.medusa_linear_w4(x.float(), q, s, z)
    with pytest.raises(ValueError, match="dense rows"):
        mg.medusa_linear_w4(x.t().contiguous().t(), q, s, z)
    with pytest.raises(mg.MedusaError, match="INVALID_ARG"):  # rows that do not start on 16 bytes
        mg.medusa_linear_w4(to_dev(bf16(rng, 4, 140))[:, 4:132], q, s, z)
    with pytest.raises(mg.MedusaError, match="INVALID_ARG"):
        mg.medusa_linear_w4(to_dev(bf16(rng, 4, 132))[:, :128], q, s, z)
    with pytest.raises(ValueError, match="y must be"):
        mg.medusa_linear_w4(x, q, s, z, y=torch.empty((4, 7), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="the stream is of|on"):
        mg.medusa_linear_w4(x, q, s.cpu(), z)


# ----------------------------------------------------------------- quantizing

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("symmetric", [False, True])
@pytest.mark.parametrize("N,K,G", [(1, 32, 32), (7, 96, 32), (33, 256, 64), (130, 512, 128), (3, 128, 128)])
def test_quantizing_is_exact(mg, N, K, G, symmetric, dtype):
    rng = np.random.default_rng(N + K)
    w = rng.standard_normal((N, K)).astype(np.float32) * 0.02
    w[0, :G] = 0.0                      # nothing: scale 1
    if N > 3:
        w[1, :G] = np.abs(w[1, :G])     # the zero is at an end
        w[2, 3], w[3, K - 1] = np.nan, -np.inf
        w[4, :G] = np.linspace(-1.0, 1.0, G) * 7  # halves
        w[5, :G] = 1e-41                # a scale that bf16 rounds to a subnormal or to 0
        w[6, :G] *= 1e30
    if dtype == "bf16":
        bits = wl.to_bf16_bits(w)
        bits[np.isnan(w)] = 0x7FC0
        bits[np.isinf(w)] = 0xFF80
        dev, w = to_dev(bits), ov.bf16_value(bits)
    else:
        dev = to_dev(w)
    q, s, z = mg.medusa_w4_quantize(dev, G, symmetric)
    eq, es, ez, bad = ov.quantize(w, G, symmetric)
    gs = ov.bf16_value(to_host(s))
    np.testing.assert_array_equal(np.isnan(gs), bad)
    np.testing.assert_array_equal(gs[~bad], es[~bad])
    ok = ~np.repeat(bad.T, G, 1)
    np.testing.assert_array_equal(ov.unpack(host_words(q))[ok], eq[ok])
    if symmetric:
        assert z is None
    else:
        np.testing.assert_array_equal(to_host(z)[~bad], ez[~bad])
    y = mg.medusa_linear_w4(torch.eye(K, dtype=torch.bfloat16, device="cuda"), q, s, z, out_dtype=torch.float32)
    want = ov.weights(host_words(q), to_host(s), None if z is None else to_host(z)).T
    fine = ~np.isnan(want).any(0)
    np.testing.assert_array_equal(value(y)[:, fine], want[:, fine])


def test_quantizing_refuses(mg):
    w = torch.zeros((4, 96), device="cuda")
    for group in (64, 16, 0, -1):
        with pytest.raises(ValueError, match="group"):
            mg.medusa_w4_quantize(w, group)
    with pytest.raises(ValueError, match="dense"):
        mg.medusa_w4_quantize(torch.zeros((4, 192), device="cuda")[:, ::2], 32)


def test_outputs_past_32_bits(mg):
    T, K, N = 70001, 64, 32016
    rng = np.random.default_rng(2)
    m, rows = matrix(rng, N, K, 64), [0, 35000, 67077, 67078, T - 1]
    x = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    few = bf16(rng, len(rows), K)
    x[rows] = to_dev(few)
    y = mg.medusa_linear_w4(x, *dev_matrix(m))
    check_linear(y[rows], few, m, "bf16")
    assert not y[1:35000].any() and not y[67079:T - 1].any()
