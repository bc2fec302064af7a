"""What the binding's dropout calls take as their counter, on a host without a
GPU: tensors are stood in for by objects that answer the same questions.  And
the keys that the documentation's example gives them."""
import os
import re

import pytest
import torch

import dropout_ref as dr


@pytest.fixture(scope="module")
def lib():
    from layernorm_fwd_bwd_b200 import build
    build.build()
    from layernorm_fwd_bwd_b200 import ln
    return ln


class Counter:
    """A tensor of `numel` elements on device `index`."""

    def __init__(self, dtype, numel=1, index=0, cuda=True):
        self.dtype, self._numel, self.is_cuda = dtype, numel, cuda
        self.device = torch.device("cuda", index) if cuda else torch.device("cpu")

    def get_device(self):
        return self.device.index if self.is_cuda else -1

    def element_size(self):
        return self.dtype.itemsize

    def numel(self):
        return self._numel

    def data_ptr(self):
        return 4096


@pytest.fixture(autouse=True)
def device_zero(monkeypatch, lib):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(lib, "_counter_types", (), raising=False)
    monkeypatch.setattr(lib, "_current_device", None, raising=False)


@pytest.mark.parametrize("counter", [
    Counter(torch.float64), Counter(torch.complex64), Counter(torch.int32, 2),
    Counter(torch.int64, 2), Counter(torch.int64, 0), Counter(torch.int64, index=1),
    Counter(torch.int64, cuda=False)],
    ids=["float64", "complex64", "int32", "two", "none", "other device", "host"])
def test_other_counters_are_refused(lib, counter):
    with pytest.raises(TypeError):
        lib._step(counter)
    # and by a whole call, before the library sees it (an n of -1 would raise
    # LNError there)
    with pytest.raises(TypeError):
        lib.ln_dropout(4096, 8192, -1, 0.1, 0, 0, counter, lib.LN_F32, stream=0)


def test_counters(lib):
    assert lib._step(None) is None
    assert lib._step(1 << 40) == 1 << 40
    for dtype in (torch.int64, torch.uint64):
        assert lib._step(Counter(dtype)) == 4096


def test_documented_keys_draw_a_mask_once():
    """README's example: over sites and steps no two dropouts have the same
    seed and offset + step, so no mask is drawn twice."""
    readme = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
    line = re.search(r"^keys = (\(.*?\))\s+#", open(readme).read(), re.M).group(1)
    drawn, masks = set(), set()
    sites, steps = 25, (0, 1, 2, 3, 10 ** 6)
    for site in range(sites):
        for step in steps:
            p, seed, offset, counter = eval(line, {"seed": 7, "site": site, "step": step})
            assert counter == step and 0 < p < 1
            drawn.add((seed, (offset + counter) % (1 << 64)))
            masks.add(dr.keep(256, p, seed, offset, counter).tobytes())
    assert len(drawn) == sites * len(steps) == len(masks)
