"""Attention over a cache of latent rows against the attention of the heads that it stands for."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    yield


@pytest.mark.parametrize("fmt,most", [(None, 2.0 ** -6), ("e4m3fn", 2.0 ** -3)])
def test_the_layer_gives_its_heads_attention(fmt, most):
    """Heads of 128 + 64 dims, whose keys are an up-projection of the latent rows beside the rotary dims: their softmax of
    q k / sqrt(192) in 64 bits, and the layer's with the up-projection in the queries. The projection has one 1 or -1 a
    latent dim, so that the queries that carry it are exact. (With the rows' 576 dims in the scale the outputs are 0.5 off.)
    Bounds: 16-bit rows, queries' rotary dims and weights are a few roundings of 2^-9 (rms); codes 2^-5 (rms) as keys and as values."""
    from fp8_quant_gb300.examples import latent_layer as ex
    H, N, R, L, n = 8, 128, 64, 512, 300
    g = torch.Generator(device="cuda").manual_seed(7)
    rows = torch.randn(n, L + R, generator=g, device="cuda").to(torch.bfloat16)
    heads = torch.randn(n, H, N + R, generator=g, device="cuda").to(torch.bfloat16)
    up = torch.zeros(H, N, L, dtype=torch.float64, device="cuda")
    sign = torch.randint(0, 2, (H, L), generator=g, device="cuda").double() * 2 - 1
    up[:, torch.arange(L, device="cuda") % N, torch.arange(L, device="cuda")] = sign
    layer = ex.LatentLayer(H, L, R, head_dim=N + R, pages=20, page_size=16, max_position=n, fmt=fmt)
    q = torch.cat((torch.einsum("thn,hnl->thl", heads[..., :N].double(), up).to(torch.bfloat16), heads[..., N:]), -1)
    table = layer.admit([n])
    got = layer.prefill(rows, q, table, [n]).double()

    def rotate(x, c, s):
        a, b = x.split(R // 2, -1)
        return torch.cat((a * c - b * s, b * c + a * s), -1)

    c, s = layer.cos_sin[:n].double().split(R // 2, -1)
    keys = torch.cat((torch.einsum("hnl,tl->htn", up, rows[:, :L].double()),
                      rotate(rows[:, L:].double(), c, s).expand(H, n, R)), -1)
    qs = torch.cat((heads[..., :N].double(), rotate(heads[..., N:].double(), c[:, None], s[:, None])), -1)
    score = torch.einsum("thd,hkd->htk", qs, keys) / (N + R) ** 0.5
    score = score.masked_fill(torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1), float("-inf"))
    want = torch.einsum("htk,kl->thl", score.softmax(-1), rows[:, :L].double())
    off = (got - want).square().sum().sqrt() / want.square().sum().sqrt()
    assert off.item() <= most
