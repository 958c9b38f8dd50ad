"""NaN blocks (scale byte 255) through the MX product and the mixture-of-experts
layer: every output that uses one is NaN, and no other.  Masks are compared, so
there is no tolerance."""
import pytest
import torch

from q4_packed_weight_amd import binding
from gpu_util import DEV
from test_mx_paths_gpu import TYPES, Layer, gen, odd, packed

pytestmark = pytest.mark.gpu


def product(a, fmt, w, M, K, N, kind):
    y = torch.zeros(M, N, dtype=TYPES[kind], device=DEV)
    binding.mxfp4_matmul(*a, fmt, *w, M, K, N, y)
    return y.isnan()


# Few tokens, 64x64, 128x128 and 256x256 tiles; an odd and an even number of
# whole 128-position steps in a row, and rows that end within one.
SIZES = [(1, 70), (20, 100), (40, 100), (65, 100), (128, 200), (300, 77), (64, 8200), (1024, 4096),
         (4096, 4096)]


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("K", [128, 256, 384, 1152, 1056])
@pytest.mark.parametrize("M,N", SIZES)
def test_product_nan_blocks_stay_in_their_row(M, N, K, fmt, kind):
    """The first four blocks of a row lie right behind the scales of the row
    before it, and the last ones right before the next row's."""
    g = gen(M, N, K, fmt)
    (ac, as_), (wc, ws) = packed(g, M, K, fmt), packed(g, N, K, "fp4")
    for blocks in ((0, 3), (3, 0), (K // 32 - 1, 1)):
        a_s, w_s = as_.clone(), ws.clone()
        rows_a, rows_w = sorted({M // 2, M - 1}), sorted({N // 3, N - 1})
        for t in rows_a:
            a_s[t, blocks[0]] = 255
        for o in rows_w:
            w_s[o, blocks[1]] = 255
        want = torch.zeros(M, N, dtype=torch.bool, device=DEV)
        want[rows_a] = True
        want[:, rows_w] = True
        assert torch.equal(product((ac, a_s), fmt, (wc, w_s), M, K, N, kind), want), blocks


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("K", [128, 384, 1056])
@pytest.mark.parametrize("M,N", SIZES)
def test_product_of_rows_quantised_with_infinities(M, N, K, fmt):
    """mx_quantize gives a block that holds a NaN or an infinity the scale byte
    255 and codes of zero: the product shows it all the same."""
    g = gen("quantised", M, N, K, fmt)

    def blocks(rows, f, at, col, value):
        x = torch.randn(rows, K, generator=g, device=DEV)
        x[at, col] = value
        codes = torch.empty(rows, K * (4 if f == "fp4" else 8) // 8, dtype=torch.uint8, device=DEV)
        scales = torch.empty(rows, K // 32, dtype=torch.uint8, device=DEV)
        binding.mx_quantize(x, rows, K, f, codes, scales)
        assert not bool(codes.view(rows, K // 32, -1)[at, col // 32].any())
        return codes, scales

    a = blocks(M, fmt, M // 2, 5, float("-inf"))
    w = blocks(N, "fp4", N // 3, K - 1, float("nan"))
    want = torch.zeros(M, N, dtype=torch.bool, device=DEV)
    want[M // 2] = want[:, N // 3] = True
    assert torch.equal(product(a, fmt, w, M, K, N, "bf16"), want)


@pytest.mark.parametrize("zero_codes", [False, True])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("T,H,F,E,k", [(1, 256, 96, 8, 2), (1, 288, 128, 8, 2), (6, 384, 160, 8, 2),
                                       (12, 128, 384, 16, 3), (40, 160, 64, 6, 2),
                                       (24, 4096, 4096, 16, 2)])
def test_expert_nan_blocks_reach_the_tokens_that_chose_it(T, H, F, E, k, kind, zero_codes):
    layer = Layer(T, H, F, E, k, kind)
    logits = layer.x.double() @ layer.router.double().t().contiguous() + layer.bias.double()
    top, order = torch.sort(logits, dim=-1, descending=True, stable=True)
    sure = top[:, k - 1] - top[:, k] > 1e-4  # far beyond what fp32 logits are off by
    e = int(order[int(sure.nonzero()[0]), k - 1])  # chosen by one token, and by which others
    chose = (order[:, :k] == e).any(-1)
    up_c, up_s = layer.up[0].view(E, 2 * F, H // 2), layer.up[1].view(E, 2 * F, H // 32)
    dn_c, dn_s = layer.down[0].view(E, H, F // 2), layer.down[1].view(E, H, F // 32)
    clean = [t.clone() for t in layer.up + layer.down]
    for codes, scales, row, block in ((up_c, up_s, F // 2, 0), (up_c, up_s, 2 * F - 1, H // 32 - 1),
                                      (dn_c, dn_s, 0, F // 32 - 1), (dn_c, dn_s, H - 1, 0)):
        for t, c in zip(layer.up + layer.down, clean):
            t.copy_(c)
        scales[e, row, block] = 255
        if zero_codes:
            codes[e, row, 16 * block:16 * block + 16] = 0
        want = torch.zeros(T, H, dtype=torch.bool, device=DEV)
        if codes is up_c:
            want[chose] = True  # one of h is NaN, and every output adds it
        else:
            want[chose, row] = True
        for odd_scales in (False, True):
            got = layer.run(odd_scales=odd_scales).isnan()
            assert torch.equal(got[sure], want[sure]), (row, block, odd_scales)
