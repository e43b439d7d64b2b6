"""The cache's tensors can be replaced: every later call sees the new one (CPU: the addresses
that the calls are given)."""
import pytest
import torch

NAMES = ["k_pool", "v_pool", "block_table", "pos", "mass", "seq_len", "next_pos"]


@pytest.fixture
def cache(crs, monkeypatch):
    """A cache of CPU tensors, whose calls are never launched."""
    need = crs._need

    def anywhere(t, name, dtype=None, shape=None):
        class Cuda(type(t)):
            is_cuda = True
        if isinstance(t, torch.Tensor):
            need(t.as_subclass(Cuda), name, dtype, shape)
            return t
        return need(t, name, dtype, shape)

    monkeypatch.setattr(crs, "_need", anywhere)
    return crs.KvCache.empty(2, 3, 40, D=64, page_size=16, device="cpu")


@pytest.mark.parametrize("name", NAMES)
def test_a_replaced_tensor_reaches_the_calls(cache, name):
    before = {n: getattr(cache.st, n) for n in NAMES}
    new = getattr(cache, name).clone()
    setattr(cache, name, new)
    assert getattr(cache, name) is new
    for n in NAMES:
        assert getattr(cache.st, n) == (new.data_ptr() if n == name else before[n])


@pytest.mark.parametrize("name", NAMES)
def test_only_a_tensor_of_the_same_kind_is_taken(cache, name):
    old, at = getattr(cache, name), getattr(cache.st, name)
    for bad in (old.double(), old[:1].clone(), old.new_zeros(old.shape[::-1]).movedim(0, -1)[..., :1], "x"):
        with pytest.raises((ValueError, TypeError)):
            setattr(cache, name, bad)
    assert getattr(cache, name) is old and getattr(cache.st, name) == at


def test_tracking_can_be_dropped_and_taken_up(cache):
    mass, pos = cache.mass, cache.pos
    cache.mass = cache.pos = None
    assert cache.st.mass is None and cache.st.pos is None and cache.cap == 40
    with pytest.raises(ValueError):
        cache.select(4)
    cache.mass, cache.pos = mass, pos
    assert cache.st.mass == mass.data_ptr() and cache.st.pos == pos.data_ptr()
    with pytest.raises((ValueError, TypeError)):
        cache.seq_len = None


def test_a_shallow_copy_keeps_its_own_addresses(cache):
    import copy
    other = copy.copy(cache)
    other.mass = cache.mass.clone()
    assert cache.st.mass == cache.mass.data_ptr() and other.st.mass == other.mass.data_ptr()
