"""Every device entry point of the binding launches on the current device: tensors of another one, or of two, are
refused before the call (a kernel that follows their pointers would read memory that its device cannot reach)."""
import pytest
import torch

import mla_paged_latent_gb300 as mla


class On:
    """A tensor as far as the binding looks before its call: it claims to live on a device."""
    is_cuda = True
    shape = (2, 2)
    dtype = None

    def __init__(self, d):
        self.device, self.get_device = f"cuda:{d}", lambda: d
        self.data_ptr, self.numel = (lambda: 256), (lambda: 1 << 20)


CALLS = {
    "mla_decode": lambda t: (t[0], t[1], 4, 64, t[2], t[3], 1, 1.0, t[4], t[5], 1, 1, t[6], t[7], t[8]),
    "mla_sparse_prefill": lambda t: (t[0], t[1], t[2], 1.0, t[3], t[4], 1, 1, t[5], t[6], t[7], t[8]),
    "mla_swa_plan": lambda t: (t[0], 64, 1, t[1], t[2]),
    "mla_decode_runs": lambda t: (t[0], t[1], 4, 64, t[2], 8, 1, 1.0, t[3], t[4], 1, 1, t[5], t[6], t[7]),
    "mla_decode_static_workspace": lambda t: (t[0], t[1], 4, 64, t[2], t[3], 1, 1.0, t[4], t[5], 1, 1, t[6], t[7]),
    "mla_combine": lambda t: (t[0], t[1], t[2], 4, 2, t[3], t[4]),
    "mla_combine_v_up": lambda t: (t[0], t[1], t[2], 1, 2, t[3], t[4], t[5], t[6]),
    "mla_combine_inv_rope": lambda t: (t[0], t[1], t[2], 1, 2, t[3], t[4], t[5], t[6]),
    "mla_kv_write": lambda t: (t[0], t[1], t[2], 4, 64, t[3]),
    "mla_kv_write_norm_rope": lambda t: (t[0], t[1], t[2], t[3], 1e-6, t[4], t[5], 4, 64, t[6]),
    "mla_qkv_norm_rope": lambda t: (t[0], t[1], t[2], t[3], t[4], t[5], 1e-6, t[6], t[7], t[8], 4, 64),
    "mla_kv_read": lambda t: (t[0], 4, 64, t[1], t[2], t[3]),
    "mla_kv_gather": lambda t: (t[0], 4, 64, t[1], 3, t[2]),
}


@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_another_device_are_refused(name, monkeypatch):
    class Lib:
        def __getattr__(self, entry):
            raise AssertionError(f"{entry} was reached")

    monkeypatch.setattr(mla, "load", lambda path=None: Lib())
    monkeypatch.setattr(mla, "_stream", lambda s: None)
    monkeypatch.setattr(mla, "_torch_c", None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    call, args = getattr(mla, name), CALLS[name]
    with pytest.raises(ValueError, match="current device"):
        call(*args([On(1)] * 9))
    used = args(list(range(100, 109)))
    for i in [x - 100 for x in used if isinstance(x, int) and x >= 100]:
        tensors = [On(0)] * 9
        tensors[i] = On(1)
        with pytest.raises(ValueError, match="one device|current device"):
            call(*args(tensors))


@pytest.mark.parametrize("name", ["mla_combine_v_up", "mla_combine_inv_rope"])
def test_partials_left_out(name, monkeypatch):
    """No partials: the other tensors are looked at all the same."""
    monkeypatch.setattr(mla, "_torch_c", None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="current device"):
        getattr(mla, name)(*CALLS[name]([None, None] + [On(1)] * 7))
