"""CPU: the cache object checks its tensors at every call, not only when it is
made.  Its own checks run on CPU tensors here (device index -1, as CPU tensors
report it); no call reaches the library."""
import pytest
import torch

from medusa_head_speculative_02_b200 import api

NAMES = ("k_codes", "k_par", "v_codes", "v_par")


def _cache(lead=(2, 3, 8), dh=64):
    mk = lambda n, dt: torch.zeros(*lead, n, dtype=dt)  # noqa: E731
    with pytest.MonkeyPatch.context() as m:
        m.setattr(api, "_need", lambda *a: None)  # (a CUDA tensor)
        return api.PackedCache(mk(dh // 2, torch.uint8), mk(2, torch.bfloat16),
                               mk(dh // 2, torch.uint8), mk(2, torch.bfloat16))


def test_sizes_and_addresses():
    c = _cache()
    assert (c.B, c.Hkv, c.Lcap, c.dh, c.layers) == (2, 3, 8, 64, None)
    assert list(c._ptrs) == [getattr(c, n).data_ptr() for n in NAMES]
    assert _cache((4, 2, 3, 8), 128).layers == 4
    c.k_par.data = torch.ones_like(c.k_par)          # other memory, same shape: followed
    assert c._ptrs[1] == c.k_par.data_ptr()


@pytest.mark.parametrize("name", NAMES)
def test_a_tensor_that_changed_is_refused(name):
    def changed(how):
        c = _cache()
        t = getattr(c, name)
        t.data = how(t)
        with pytest.raises((ValueError, TypeError)):
            c._ptrs
    changed(lambda t: t[:1].clone())                           # fewer sequences
    changed(lambda t: t[:, :, :4].clone())                     # a smaller capacity
    changed(lambda t: t[:, :, :4])                             # a strided view
    changed(lambda t: t.transpose(0, 1).contiguous().transpose(0, 1))
    changed(lambda t: t.new_zeros(2, 3, 8, 2 * t.shape[-1])[..., ::2])


@pytest.mark.parametrize("name", NAMES)
def test_a_resized_tensor_is_refused(name):
    c = _cache()
    getattr(c, name).resize_(1, 3, 8, getattr(c, name).shape[-1])
    with pytest.raises(ValueError, match=name):
        c._ptrs


@pytest.mark.parametrize("name", NAMES + ("B", "Hkv", "Lcap", "dh", "layers", "device"))
def test_sizes_and_tensors_are_read_only(name):
    c = _cache()
    with pytest.raises(AttributeError):
        setattr(c, name, 1)
