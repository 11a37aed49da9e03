"""Calls of the 8-bit projections that their first tests do not make."""

import pytest

import invariant_mmdit_joint_gb300 as pkg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    return d


def test_turned_operands_past_32_bits(dev):
    """Gradients of 270000 tokens, whose turned codes (8192 x 270000 bytes, x's and dy's) and gradients have places past
    2^31. dy is 0 but for the last 300 tokens: dw and db are those of the last 688 alone, which start where a sum's chunk
    of 512 tokens and a column sum's run of 8 x 128 do, and dx's last rows too; every byte."""
    import torch
    rows, some, live, n = 270000, 688, 300, 8192
    assert (rows - some) % 1024 == 0 and n * rows > 1 << 31
    g = torch.Generator(device=dev)
    g.manual_seed(6)
    x = torch.full((1, rows, n), 0.5, dtype=torch.bfloat16, device=dev)
    dy = torch.zeros_like(x)
    x[0, -some:] = torch.randn((some, n), generator=g, device=dev).bfloat16()
    dy[0, -live:] = (1e-3 * torch.randn((live, n), generator=g, device=dev)).bfloat16()
    w = (torch.randn((n, n), generator=g, device=dev) / n ** 0.5).bfloat16()
    got = []
    for t in (some, rows):
        op = pkg.Fp8Projection(1, 0, t, n, n, device=dev, grad_format="e5m2")
        op.set_weights((None, w))
        f = op.forward((None, x[:, -t:].contiguous()), train=True)
        codes = f["xt"][1].view(torch.uint8)
        assert codes.numel() > 1 << 31 or t == some
        r = op.backward((None, dy[:, -t:].contiguous()), f)
        pkg.rlk_joint_attn_check_status()
        first = -(-t // 16) * 16 - some  # of the tokens' codes in a row
        got.append([f["y"][1][0, -live:].clone(), codes[:, first:first + some].clone(), r["dw"][1], r["db"][1],
                    r["dx"][1][0, -live:].clone()])
        assert bool((r["dx"][1][0, :t - some] == 0).all())
        del op, f, r, codes
        torch.cuda.empty_cache()
    assert float(got[0][2].abs().max()) > 0 and all(bool(torch.equal(a.view(torch.uint8), b.view(torch.uint8))) for a, b in zip(*got))
