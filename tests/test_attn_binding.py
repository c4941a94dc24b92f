"""Which tensors the attention-side binding takes, without a GPU: host tensors that say they are on one, and a library that
notes every call instead of making it."""
import types

import pytest
import torch

from weight_only_int4_route_gb300 import attn

BF16 = torch.bfloat16


class Fake(torch.Tensor):
    """A host tensor that says it is on GPU `on`."""
    on = 0
    is_cuda = True

    def get_device(self):
        return self.on


class Fake1(Fake):
    on = 1


def on(t, dev=0):
    return t.as_subclass(Fake1 if dev else Fake)


def ints(*v, dev=0):
    return on(torch.tensor(v, dtype=torch.int32), dev)


@pytest.fixture
def calls(monkeypatch):
    """The library calls made, (name, arguments) each.  GPU 0 is current."""
    made = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: made.append((name, a)) or 0

    monkeypatch.setattr(attn, "lib", Library)
    monkeypatch.setattr(attn, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(attn, "_current_device", lambda: 0, raising=False)
    return made


def setup(dev=0, cache_dev=0, heads=2):
    D = 16
    s = types.SimpleNamespace()
    s.cache = attn.KVCache(on(torch.zeros((2, 4, 2, heads, 8, D), dtype=BF16), cache_dev), ints(*[-1] * 6, dev=cache_dev).reshape(2, 3),
                           ints(0, 0, dev=cache_dev), ints(0, 0, 0, 0, dev=cache_dev))
    s.x, s.q = (on(torch.zeros((3, h, D), dtype=BF16), dev) for h in (heads, 2 * heads))
    s.pos, s.cu, s.seqs, s.start = ints(0, 1, 2, dev=dev), ints(0, 3, dev=dev), ints(0, dev=dev), ints(0, dev=dev)
    s.table = on(torch.zeros((8, D)), dev)
    return s


CALLS = {
    "rope": lambda s: attn.rope(s.x, s.pos, s.table),
    "rope_out": lambda s: attn.rope(s.x, s.pos, s.table, out=s.x),
    "extend": lambda s: s.cache.extend(s.seqs, s.start),
    "fork": lambda s: s.cache.fork(s.seqs, s.start),
    "free": lambda s: s.cache.free(s.seqs),
    "compact": lambda s: s.cache.compact(s.seqs, s.start, s.cu[:2], s.pos),
    "copy": lambda s: s.cache.copy(s.seqs, s.start),
    "append": lambda s: s.cache.append(s.x, s.x, s.cu, s.seqs, s.start),
    "append_rotated": lambda s: s.cache.append(s.x, s.x, s.cu, s.seqs, s.start, q=s.q, pos=s.pos, cos_sin=s.table),
    "tree_mask": lambda s: attn.tree_mask(s.pos, s.cu, s.start, 4),
    "attention": lambda s: attn.attention(s.q, s.cache, s.cu, s.seqs, s.start),
    "masked": lambda s: attn.attention(s.q, s.cache, s.cu, s.seqs, s.start, mask=s.pos.reshape(3, 1)),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_tensors_on_the_current_gpu_are_taken(calls, name):
    CALLS[name](setup())
    assert calls


@pytest.mark.parametrize("name", sorted(CALLS))
def test_tensors_on_another_gpu_are_refused(calls, name):
    """The library launches on the current GPU: its kernels must not be given another one's addresses."""
    s = setup(dev=1, cache_dev=1)
    with pytest.raises(AssertionError):
        CALLS[name](s)
    assert not calls


@pytest.mark.parametrize("name", sorted(set(CALLS) - {"rope", "rope_out", "tree_mask"}))
@pytest.mark.parametrize("dev", [0, 1])
def test_a_cache_on_another_gpu_than_its_arguments_is_refused(calls, name, dev):
    s = setup(dev=dev, cache_dev=1 - dev)
    with pytest.raises(AssertionError):
        CALLS[name](s)
    assert not calls


@pytest.mark.parametrize("name,field", [("rope", "x"), ("rope", "pos"), ("rope", "table"), ("extend", "start"), ("fork", "start"),
                                        ("copy", "seqs"), ("compact", "pos"), ("append", "cu"), ("append", "x"),
                                        ("append_rotated", "pos"), ("append_rotated", "table"), ("append_rotated", "q"),
                                        ("tree_mask", "start"), ("attention", "q"), ("attention", "cu"), ("masked", "pos")])
def test_one_tensor_on_another_gpu_is_refused(calls, name, field):
    s = setup()
    setattr(s, field, getattr(s, field).as_subclass(Fake1))
    with pytest.raises(AssertionError):
        CALLS[name](s)
    assert not calls


def test_parts_of_a_cache_on_two_gpus_are_refused(calls):
    s = setup().cache
    with pytest.raises(AssertionError):
        attn.KVCache(s.pool, s.table, s.lens.as_subclass(Fake1), s.refs)
    with pytest.raises(AssertionError):
        attn.KVCache(s.pool.as_subclass(Fake1), s.table, s.lens, s.refs)


def test_a_rotary_table_on_another_gpu_is_refused(calls, monkeypatch):
    monkeypatch.setattr(attn.torch, "empty", lambda *a, **k: on(torch.zeros(4), 1))
    with pytest.raises(AssertionError):
        attn.rope_table(2, 2)
    assert not calls


def odd(t):
    """t with a stride of 5 in every dimension of one."""
    return t.as_strided(t.shape, [5 if n == 1 else s for n, s in zip(t.shape, t.stride())])


@pytest.mark.parametrize("name", ["rope", "rope_out", "append_rotated", "attention"])
def test_the_stride_of_a_single_head_is_open(calls, name):
    s = setup(heads=1)
    CALLS[name](s)
    plain = list(calls)
    s.x = odd(s.x)
    calls.clear()
    CALLS[name](s)
    strides = {"moe_rope": slice(3, 7)}
    for (n0, a0), (n1, a1) in zip(plain, calls):
        assert n0 == n1 and a0[strides.get(n0, slice(0))] == a1[strides.get(n0, slice(0))]
