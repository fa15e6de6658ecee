"""A cache whose tensors lie on more than one device is refused before its pointers are taken (no
GPU: tensors that only know their shape, type and device)."""
import pytest
import torch

import query_aware_kv_gb300 as q
from query_aware_kv_gb300 import _lib


class Elsewhere:
    def __init__(self, shape, device):
        self.shape, self.device = torch.Size(shape), device

    def get_device(self):
        return self.device

    def data_ptr(self):
        return 256


NARROW = dict(k_pool=(9, 2, 16, 128), v_pool=(9, 2, 16, 128), k_scale=(9, 2), v_scale=(9, 2),
              k_open=(3, 2, 16, 128), v_open=(3, 2, 16, 128), meta=(3, 2, 4, 2, 128),
              block_table=(3, 4), seq_lens=(3,))
PAGED = {n: NARROW[n] for n in ("k_pool", "v_pool", "meta", "block_table", "seq_lens")}


@pytest.mark.parametrize("make,shapes", [(q.NarrowCache, NARROW), (q.PagedCache, PAGED)],
                         ids=["narrow", "paged"])
def test_every_tensor_of_a_cache_is_on_its_device(monkeypatch, make, shapes):
    monkeypatch.setattr(_lib, "_need", lambda *a, **k: None)

    def cache(**devices):
        return make(num_q_heads=4, **{n: Elsewhere(s, devices.get(n, 1)) for n, s in shapes.items()})

    assert cache().batch == 3
    for name in shapes:
        with pytest.raises(ValueError, match="another device"):
            cache(**{name: 0})


@pytest.mark.parametrize("plan,calls", [(q.NarrowPlan, ("decode", "dense", "step")), (q.WindowPlan, ("decode",)),
                                        (q.DecodePlan, ("decode", "step"))])
def test_a_plan_is_not_launched_on_another_device(monkeypatch, plan, calls):
    """A plan made on device 0, called while device 1 is the current one."""
    monkeypatch.setattr(_lib, "_current_device", lambda: 1)
    p = object.__new__(plan)
    p._dev, p._many = 0, True
    for name in calls:
        with pytest.raises(ValueError, match="current"):
            getattr(p, name)(*[None] * (3 if name == "step" else 1))
