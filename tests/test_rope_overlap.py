"""Which outputs a rope call accepts: the check of addresses and strides, on views of
CPU buffers (nothing is launched), against the addresses of every element."""

import itertools

import numpy as np
import pytest
import torch

import block_sparse_attention_bwd_b200 as sp


def _triple(t):
    return t.data_ptr(), t.shape, t.stride()


def _refused(ins, outs):
    try:
        sp._rope_overlaps("rope", [_triple(t) for t in ins], [_triple(t) for t in outs], ins[0].element_size())
    except ValueError:
        return True
    return False


def _addresses(t):
    at = np.array(t.data_ptr(), np.int64)
    for n, st in zip(t.shape, t.stride()):
        at = at[..., None] + np.arange(n, dtype=np.int64) * st * t.element_size()
    return at.ravel()


def _wrong(ins, outs):
    """By definition: an output element is written twice, or is another element's input."""
    every = np.concatenate([_addresses(t) for t in outs])
    if len(np.unique(every)) != len(every):
        return True
    for i, j in itertools.product(range(len(outs)), range(len(ins))):
        a, b = _addresses(outs[i]), _addresses(ins[j])
        if i == j and (a == b).all():
            continue  # in place
        if np.intersect1d(a, b).size:
            return True
    return False


def _check(ins, outs, refused):
    assert _wrong(ins, outs) == refused
    assert _refused(ins, outs) == refused


def _packed(B=2, S=6, H=7, D=8, pad=0):
    buf = torch.zeros((B, S, H, D + pad))
    return lambda a, b: buf[:, :, a:b, :D].transpose(1, 2)


def test_outputs_that_share_heads_are_refused():
    ins = [torch.zeros(2, 4, 6, 8) for _ in range(2)]
    heads = _packed()
    _check(ins, [heads(0, 4), heads(2, 6)], True)
    buf = torch.zeros(2, 7, 6, 8)
    _check(ins, [buf[:, :4], buf[:, 2:6]], True)
    _check(ins, [buf[:, 3:7], buf[:, :4]], True)
    _check([ins[0], ins[1][:, :3]], [buf[:, 3:7], buf[:, :3]], False)
    _check([ins[0], ins[1][:, :3]], [heads(3, 7), heads(0, 3)], False)


def test_in_place_of_one_input_only():
    """Q in place and K to a new tensor (or the other way round), both views of one packed buffer."""
    heads = _packed()
    q, k, v = heads(0, 4), heads(4, 6), heads(6, 7)
    other = torch.zeros(2, 2, 6, 8)
    _check([q, k], [q, other], False)
    _check([q, k], [torch.zeros(2, 4, 6, 8), k], False)
    _check([q, k], [q, k], False)
    _check([heads(0, 1), heads(1, 2)], [heads(1, 2), heads(0, 1)], True)  # swapped
    _check([heads(0, 1), heads(1, 2)], [heads(2, 3), heads(6, 7)], False)  # into unused heads of the same buffer
    _check([v, v], [v, heads(0, 1)], True)  # K would read what Q writes
    _check([q], [heads(1, 5)], True)


def test_an_output_that_overlaps_itself():
    q = torch.zeros(1, 2, 5, 8)
    base = torch.zeros(400)
    _check([q], [base.as_strided((1, 2, 5, 8), (0, 40, 8, 1))], False)
    _check([q], [base.as_strided((1, 2, 5, 8), (0, 40, 4, 1))], True)  # rows closer than their length
    _check([q], [base.as_strided((1, 2, 5, 8), (0, 32, 8, 1))], True)  # a head that starts inside the one before
    _check([q], [base.as_strided((1, 2, 5, 8), (7, 0, 8, 1))], True)
    _check([q], [base.as_strided((1, 2, 5, 8), (7, 8, 16, 1))], False)  # heads between each other's rows
    _check([torch.zeros(2, 2, 5, 8)], [base.as_strided((2, 2, 5, 8), (24, 8, 16, 1))], True)


def test_halves_of_wider_rows():
    wide = torch.zeros(2, 3, 6, 32)
    a, b = wide[..., :16], wide[..., 16:]
    _check([a, b], [a, torch.zeros(2, 3, 6, 16)], False)
    _check([a, a.clone()], [b, a], True)  # K's output is Q's input
    _check([a, a.clone()], [b, torch.zeros_like(a)], False)
    _check([a], [wide[..., 8:24]], True)


@pytest.mark.parametrize("seed", range(12))
def test_against_the_addresses_of_every_element(seed):
    """Random views of one buffer, strides nested or not: never accepted when wrong, and refused without need only
    where the search gives up (which these sizes never make it do)."""
    rng = np.random.default_rng(seed)
    base = torch.zeros(4096)
    counts = [0, 0]
    for _ in range(60):
        def view(heads, shape):
            dims = [shape[0], heads, shape[1]]
            order, st = rng.permutation(3), [0, 0, 0]
            step = shape[2] + int(rng.integers(0, 5))
            for i in order:
                st[i] = step if rng.random() < 0.9 else int(rng.integers(0, 2 * step + 1))
                step = max(step, st[i] * dims[i]) + int(rng.integers(0, 3)) * shape[2]
            return base.as_strided((dims[0], dims[1], dims[2], shape[2]), (*st, 1), int(rng.integers(0, 200)))
        shape = (int(rng.integers(1, 3)), int(rng.integers(1, 5)), int(rng.integers(1, 9)))
        heads = [int(rng.integers(1, 5)) for _ in range(2)]
        ins = [view(h, shape) if rng.random() < 0.5 else torch.zeros(shape[0], h, shape[1], shape[2]) for h in heads]
        outs = [t if rng.random() < 0.3 else view(h, shape) for t, h in zip(ins, heads)]
        wrong = _wrong(ins, outs)
        counts[wrong] += 1
        assert _refused(ins, outs) == wrong, [_triple(t) for t in ins + outs]
    assert min(counts) > 3
