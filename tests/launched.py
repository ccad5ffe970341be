"""Which kernels a call launches, by torch's own record of them."""
import warnings


def kernels(call):
    """Names of the kernels that ``call`` launches, in order, from the template's name on: "f<1, 2>". None where the
    record is empty (no tracer on this machine)."""
    import torch
    from torch.profiler import ProfilerActivity, profile
    torch.cuda.synchronize()
    with warnings.catch_warnings():
        warnings.simplefilter("ignore")
        with profile(activities=[ProfilerActivity.CUDA]) as p:
            call()
            torch.cuda.synchronize()
        events = [e for e in p.events() if e.device_type == torch.autograd.DeviceType.CUDA and "moe::" in e.name]
    events.sort(key=lambda e: e.time_range.start)
    return [e.name.split("moe::", 1)[1].split("(")[0] for e in events] or None


def assert_launched(call, *want):
    """Each name of ``want`` is the beginning of the next kernel that ``call`` launches, which are no more."""
    got = kernels(call)
    if got is None:
        warnings.warn("no record of the launched kernels: which ones ran was not checked")
        return
    assert len(got) == len(want) and all(g.startswith(w) for g, w in zip(got, want)), got
