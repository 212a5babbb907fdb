"""Windows over nodes deeper than they are long: a chain whose masks name the last nodes of its path sees what the causal windowed rows
see; whole paths stay seen."""
import numpy as np
import pytest
import torch

from tests import kv4_ref as ref, tree_ref as tr
from tests.test_gpu_kv4 import Case
from tests.test_gpu_tree import Tree


def last(masks, window):
    """Of each mask the last `window` nodes."""
    out = []
    for m in masks:
        bits = [i for i in range(m.bit_length()) if m >> i & 1]
        out.append(sum(1 << i for i in bits[-window:]))
    return out


@pytest.mark.parametrize("window", [1, 2, 5, 20, 39, 40, 41, 100])
def test_what_the_masks_of_the_last_nodes_see(window):
    T, n = 70, 40
    masks = tr.masks(list(range(-1, n - 1)))
    causal = ref.seen(T, n, True, window)
    assert np.array_equal(tr.seen(T, T - n, last(masks, window), 1, window), causal)
    whole = tr.seen(T, T - n, masks, 1, window)
    deep = np.arange(n) >= window  # as many ancestors as the window has places, or more
    assert np.array_equal(whole[~deep], causal[~deep]) and (whole[deep].sum(1) > causal[deep].sum(1)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("window", [1, 7, 16, 33, 64])
@pytest.mark.parametrize("G,n,dtype", [(2, 9, "bf16"), (4, 40, "fp16"), (8, 40, "bf16"), (1, 200, "fp16")])
def test_chains_within_a_window(window, G, n, dtype):
    args = dict(Hkv=2, G=G, D=64, P=16, dtype=dtype, seed=n + window)
    c, plain = Tree([300, n + 3, n], [n, n, n], chain=True, **args), Case([300, n + 3, n], [n, n, n], **args)
    cut = [last(ms, window) for ms in c.masks]
    out, lse = c.check(window=window, masks=cut)
    c.check(window=window)  # whole paths, as the statement has them
    rows, rl = plain.check(window=window)
    torch.cuda.synchronize()
    # the same values (below 5): two roundings to BF16, three to FP16 of each side's weights and values
    assert (rl - lse).abs().max() < 1e-3
    assert ((rows.float() - out.float()).abs() <= 2 * 2.0 ** -8 * rows.float().abs() + 6 * 2.0 ** -11 * 5).all()
