"""What an exact product shows: on the oracle's side, a block of k that is
missing, doubled or taken from its neighbour changes the bf16 results that are
compared, at the largest K as well."""
import pytest
import torch

from tests.exact_products import W_MAX, integers, product


@pytest.mark.parametrize("T,K,n", [(1, 32768, 64), (1, 32784, 160), (16, 4128, 64), (1100, 32768, 64)])
def test_a_wrong_block_shows(T, K, n):
    g = torch.Generator().manual_seed(K + T)
    x = integers((min(T, 64), K), g, device="cpu")
    codes = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6])
    W = codes[torch.randint(0, 8, (K, n), generator=g)] * torch.randint(1, 3, (K // 16, 1, 1), generator=g).expand(
        -1, 16, n).reshape(K, n) * (torch.randint(0, 2, (K, n), generator=g) * 2 - 1)
    assert W.abs().max() == W_MAX
    want = product(x, W)
    for k in (0, K // 2 // 32 * 32, K - 32):
        for change in ("missing", "doubled", "neighbour"):
            V = W.clone()
            if change == "missing":
                V[k:k + 32] = 0
            elif change == "neighbour":
                V[k:k + 32] = W[(k + 32) % (K - 31):][:32]
            a = x
            if change == "doubled":
                V, a = torch.cat((W, W[k:k + 32])), torch.cat((x, x[:, k:k + 32]), 1)
            assert not torch.equal(product(a, V), want), (k, change)


def test_every_partial_sum_is_exact():
    """Sums of 32,768 products in fp32, forwards, backwards and in a tree, are the sum in 64 bits."""
    g = torch.Generator().manual_seed(0)
    a = integers((32768,), g, device="cpu").float()
    b = torch.randint(-24, 25, (32768,), generator=g).float() / 2
    p = a * b
    want = p.double().sum()
    assert p.cumsum(0)[-1] == want and p.flip(0).cumsum(0)[-1] == want and p.view(-1, 16).sum(1).view(-1, 2).sum() == want
