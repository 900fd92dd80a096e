"""Host side of the AdamW step and the gradient norm: defaults, validation, refusals of the
Python front end (no GPU needed; validation errors are raised before any HIP call). Calls that
pass fake device addresses run only where no GPU is present."""
import ctypes
import math
import os
import subprocess

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import orthogonalized_momentum_optimizer_amd as om
from orthogonalized_momentum_optimizer_amd import _lib as L

no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(),
                                 reason="fake device addresses are only used without a GPU")
BF16, F32 = L.MUON_DT_BF16, L.MUON_DT_F32
BASE = 1 << 40                                   # fake device addresses, never dereferenced


def entries(state=L.MUON_ADAMW_8BIT):
    """Three tensors of 1000, 0 and 4096 elements, 1 MiB between buffers."""
    out, at = [], BASE
    for i, n in enumerate((1000, 0, 4096)):
        ptr = [at + (k << 20) for k in range(6)]
        at += 8 << 20
        e = dict(param=ptr[0], master=None if i else ptr[1], exp_avg=ptr[2], exp_avg_sq=ptr[3],
                 exp_avg_scale=ptr[4], exp_avg_sq_scale=ptr[5], numel=n, pdt=BF16, gdt=F32, wd=1.0)
        if n == 0:
            e.update(param=None, exp_avg=None, exp_avg_sq=None, exp_avg_scale=None,
                     exp_avg_sq_scale=None)
        if state == L.MUON_ADAMW_F32:
            e.update(exp_avg_scale=None, exp_avg_sq_scale=None)
        out.append(e)
    return out


def create(ents, state=L.MUON_ADAMW_8BIT, n=None):
    arr = L.make_adamw_tensors([tuple(e.values()) for e in ents])
    return L.muon_adamw_plan_create(arr, len(ents) if n is None else n, state)


def status_of(fn, *args, **kw):
    with pytest.raises(L.MuonError) as e:
        fn(*args, **kw)
    return e.value.status, str(e.value)


@pytest.mark.parametrize("state", [L.MUON_ADAMW_F32, L.MUON_ADAMW_8BIT])
def test_plan_of_legal_tensors(state):
    L.muon_adamw_plan_destroy(create(entries(state), state))
    empty = L.muon_adamw_plan_create(None, 0, state)
    L.muon_adamw_step(empty, None, 0, L.muon_adamw_config_default(), 0)   # no work, no HIP call
    L.muon_adamw_plan_destroy(empty)


def test_config_default():
    c = L.muon_adamw_config_default()
    assert [round(x, 9) for x in (c.lr, c.beta1, c.beta2, c.eps, c.weight_decay)] == [
        0.001, 0.899999976, 0.999000013, 1e-8, 0.01]
    assert (c.step, c.grad_scale, c.skip_nonfinite, c.stochastic, c.seed) == (1, None, 0, 1, 0)
    L.lib().muon_adamw_config_default(None)
    c = om.make_adamw_config(seed=-1, skip_nonfinite=True, stochastic=False, step=9)
    assert (c.step, c.skip_nonfinite, c.stochastic, c.seed) == (9, 1, 0, 2 ** 64 - 1)


INV, UNS, WS = L.MUON_ERR_INVALID_ARG, L.MUON_ERR_UNSUPPORTED, L.MUON_ERR_WORKSPACE


@pytest.mark.parametrize("change,status", [
    (dict(numel=-1), INV), (dict(numel=2 ** 35 + 1), UNS), (dict(pdt=7), INV), (dict(pdt=F32), INV), (dict(gdt=-1), INV),
    (dict(wd=math.inf), INV), (dict(wd=math.nan), INV), (dict(param=None), INV),
    (dict(exp_avg=None), INV), (dict(exp_avg_sq=None), INV), (dict(exp_avg_scale=None), INV),
    (dict(exp_avg_sq_scale=None), INV), (dict(param=BASE + 8), INV), (dict(master=BASE + 4), INV),
    (dict(exp_avg=BASE + (2 << 20) + 1), INV), (dict(exp_avg_sq=BASE + (2 << 20)), INV),
    (dict(exp_avg_scale=BASE + (2 << 20) + 999), INV),     # the last byte of exp_avg
    (dict(exp_avg_scale=BASE + (5 << 20) + 3), INV),       # its own 4 bytes meet the other scales
], ids=str)
def test_plan_rejects_tensors(change, status):
    ents = entries()
    ents[0].update(change)
    got, msg = status_of(create, ents)
    assert got == status, msg


def test_scales_need_no_alignment():
    ents = entries()
    ents[0].update(exp_avg_scale=BASE + (2 << 20) + 1000)   # right behind exp_avg
    L.muon_adamw_plan_destroy(create(ents))


def test_plan_rejects_counts_and_states():
    assert status_of(create, entries(), n=-1)[0] == INV
    assert status_of(create, entries(), n=2 ** 60)[0] == UNS
    assert status_of(create, entries(), state=2)[0] == INV
    assert status_of(L.muon_adamw_plan_create, None, 2, 0)[0] == INV
    assert L.lib().muon_adamw_plan_create(None, None, 0, 0) == INV
    L.lib().muon_adamw_plan_destroy(None)


@pytest.mark.parametrize("field,value", [
    ("lr", math.nan), ("eps", -1e-9), ("eps", math.inf), ("weight_decay", math.inf),
    ("beta1", 1.0), ("beta1", -0.1), ("beta2", 1.0), ("beta2", math.nan), ("step", 0),
    ("step", -3), ("skip_nonfinite", 2), ("stochastic", -1), ("skip_nonfinite", 1),
    ("grad_scale", BASE + 2), ("grad_scale", BASE), ("grad_scale", BASE + (8 << 21) + 8188)])
def test_step_rejects_config(field, value):
    plan = create(entries())
    cfg = L.muon_adamw_config_default()
    setattr(cfg, field, value)
    grads = L.make_pointers([None] * 3)                     # no gradient: nothing to enqueue
    status, msg = status_of(L.muon_adamw_step, plan, grads, 3, cfg, 0)
    assert status == INV, msg
    L.muon_adamw_plan_destroy(plan)


def test_step_rejects_decay_overflow_and_null():
    ents = entries()
    ents[2]["wd"] = 3e38
    plan = create(ents)
    cfg = L.muon_adamw_config_default()
    cfg.weight_decay = 10.0
    grads = L.make_pointers([None] * 3)
    assert status_of(L.muon_adamw_step, plan, grads, 3, cfg, 0)[0] == INV
    cfg.weight_decay = 0.0
    L.muon_adamw_step(plan, grads, 3, cfg, 0)               # every tensor left out: no HIP call
    assert status_of(L.muon_adamw_step, plan, grads, 2, cfg, 0)[0] == INV
    assert status_of(L.muon_adamw_step, plan, None, 3, cfg, 0)[0] == INV
    assert status_of(L.muon_adamw_step, None, grads, 3, cfg, 0)[0] == INV
    assert L.lib().muon_adamw_step(plan, grads, 3, None, 0) == INV
    L.muon_adamw_plan_destroy(plan)


@no_gpu_only
@pytest.mark.parametrize("grad", [
    BASE + (64 << 20) + 2,                                  # not 16-byte aligned
    BASE,                                                   # the parameter
    BASE + (2 << 20) - 16,                                  # its end meets exp_avg
    BASE + (4 << 20),                                       # the scales
    BASE + (16 << 20) + 8176])                              # the last elements of tensor 2
def test_step_rejects_gradients(grad):
    plan = create(entries())
    grads = L.make_pointers([grad, None, None])
    status, msg = status_of(L.muon_adamw_step, plan, grads, 3, L.muon_adamw_config_default(), 0)
    assert status == INV and "gradient 0" in msg
    L.muon_adamw_plan_destroy(plan)


def test_table():
    lib = L.lib()
    assert lib.muon_adamw_plan_table_size(None) == 0
    assert status_of(L.muon_adamw_plan_upload, None, BASE, 0, 0)[0] == INV
    empty = L.muon_adamw_plan_create(None, 0, 0)
    assert L.muon_adamw_plan_table_size(empty) == 0
    L.muon_adamw_plan_upload(empty, None, 0, 0)                    # nothing to fill: no HIP call
    L.muon_adamw_plan_destroy(empty)
    plan = create(entries())
    size = L.muon_adamw_plan_table_size(plan)
    assert 0 < size <= 256                                         # two tensors have elements
    for table, given, status in ((None, size, WS), (BASE + 8, size, WS), (BASE + (64 << 20), size - 1, WS),
                                 (BASE, size, INV), (BASE + (2 << 20) - 16, size, INV)):
        assert status_of(L.muon_adamw_plan_upload, plan, table, given, 0)[0] == status
    L.muon_adamw_plan_destroy(plan)


@no_gpu_only
def test_step_needs_the_table():
    plan = create(entries())
    grads = L.make_pointers([BASE + (64 << 20), None, None])
    status, msg = status_of(L.muon_adamw_step, plan, grads, 3, L.muon_adamw_config_default(), 0)
    assert status == WS and "upload" in msg
    L.muon_adamw_plan_destroy(plan)


# ---- gradient norm ---------------------------------------------------------------------------

def test_grad_plan_rejects():
    for numel, dtype, status in (([-1], [F32], INV), ([2 ** 35 + 1], [F32], UNS), ([4], [2], INV)):
        assert status_of(L.muon_grad_plan_create, numel, dtype)[0] == status
    lib, out = L.lib(), ctypes.c_void_p()
    one = (ctypes.c_int64 * 1)(4)
    assert lib.muon_grad_plan_create(None, one, None, 1) == INV
    assert lib.muon_grad_plan_create(ctypes.byref(out), one, None, 1) == INV
    assert lib.muon_grad_plan_create(ctypes.byref(out), None, None, -1) == INV
    assert lib.muon_grad_plan_create(ctypes.byref(out), one, (ctypes.c_int * 1)(0), 2 ** 50) == UNS
    assert out.value is None
    lib.muon_grad_plan_destroy(None)
    with pytest.raises(ValueError):
        L.muon_grad_plan_create([1], [F32, F32])


def test_grad_plan_workspace():
    assert L.muon_grad_plan_workspace_size(None) == 0
    empty = L.muon_grad_plan_create([], [])
    assert L.muon_grad_plan_workspace_size(empty) == 0
    L.muon_grad_plan_destroy(empty)
    for numel in ([1], [0, 0], [10 ** 6, 3], [2 ** 35] * 3):
        plan = L.muon_grad_plan_create(numel, [BF16] * len(numel))
        size = L.muon_grad_plan_workspace_size(plan)
        assert 0 < size <= 1 << 20                          # a bounded number of partial sums
        L.muon_grad_plan_destroy(plan)


def norm_call(mutate=lambda a: None):
    plan = L.muon_grad_plan_create([1000, 0, 64], [BF16, F32, F32])
    size = L.muon_grad_plan_workspace_size(plan)
    a = dict(plan=plan, grads=[BASE, None, BASE + (1 << 20)], n=3, max_norm=1.0, out=BASE + (2 << 20),
             norms=BASE + (3 << 20), workspace=BASE + (4 << 20), workspace_bytes=size, stream=0)
    mutate(a)
    a["grads"] = None if a["grads"] is None else L.make_pointers(a["grads"])
    try:
        return status_of(L.muon_grad_norm, **a)
    finally:
        L.muon_grad_plan_destroy(plan)


@no_gpu_only
@pytest.mark.parametrize("change,status", [
    (dict(plan=None), INV), (dict(n=2), INV), (dict(grads=None), INV), (dict(max_norm=-1.0), INV),
    (dict(max_norm=math.nan), INV), (dict(out=None), INV), (dict(workspace=None), WS),
    (dict(workspace=BASE + (4 << 20) + 8), WS), (dict(workspace_bytes=3), WS),
    (dict(out=BASE + 1992), INV), (dict(norms=BASE + (2 << 20) + 4), INV),
    (dict(out=BASE + (2 << 20) + 2), INV), (dict(norms=BASE + (3 << 20) + 1), INV),
    (dict(workspace=BASE + (3 << 20)), INV), (dict(grads=[BASE + 2, None, None]), INV)], ids=str)
def test_grad_norm_rejects(change, status):
    got, msg = norm_call(lambda a: a.update(change))
    assert got == status, msg


@no_gpu_only
def test_grad_scale_rejects():
    plan = L.muon_grad_plan_create([1000, 64], [BF16, F32])
    P = L.make_pointers
    for grads, n, scale in (([BASE, BASE + 1984], 2, BASE + 4096), ([BASE, BASE], 2, BASE + 4096),
                            ([BASE, None], 2, None), ([BASE, None], 1, BASE + 4096),
                            ([BASE + 4, None], 2, BASE + 4096), ([BASE, None], 2, BASE + 4097), ([BASE, None], 2, BASE + 1996)):
        assert status_of(L.muon_grad_scale, plan, P(grads), n, scale, 0)[0] == INV
    L.muon_grad_scale(plan, P([None, None]), 2, BASE, 0)     # nothing to do: no HIP call
    L.muon_grad_plan_destroy(plan)


# ---- the Python front end --------------------------------------------------------------------

def cpu_args(n=300, small=False):
    z = torch.zeros
    if small:
        b = -(-n // 256)
        return dict(params=[z(n)], exp_avgs=[z(n, dtype=torch.uint8).view(torch.float8_e4m3fn)],
                    exp_avg_sqs=[z(n, dtype=torch.uint8).view(torch.float8_e4m3fn)],
                    grad_dtypes=[torch.float32],
                    exp_avg_scales=[z(b, dtype=torch.uint8).view(torch.float8_e8m0fnu)],
                    exp_avg_sq_scales=[z(b, dtype=torch.uint8).view(torch.float8_e8m0fnu)])
    return dict(params=[z(n)], exp_avgs=[z(n)], exp_avg_sqs=[z(n)], grad_dtypes=[torch.float32])


def test_tensor_addresses_on_the_host():
    """The native check refuses what is not a CUDA tensor of the layout (the accepted cases are
    the GPU tests'), and buffers of another length."""
    numels, dtypes = (ctypes.c_int64 * 3)(4, 4, 4), (ctypes.c_int32 * 3)(1, 1, 1)
    out = L.tensor_addresses([None] * 3, numels, dtypes, 0)
    assert list(out) == [None] * 3
    for bad in (torch.zeros(4), torch.zeros(4, device="meta"), "text", 5, torch.zeros(4).to_sparse()):
        assert L.tensor_addresses([None, bad, None], numels, dtypes, 0) == 1
        assert L.tensor_addresses((bad, None, None), numels, dtypes, 0) == 0
    with pytest.raises(ValueError):
        L.tensor_addresses([None] * 2, numels, dtypes, 0)
    with pytest.raises(TypeError):
        L.tensor_addresses(7, numels, dtypes, 0)


def test_tensors_without_storage():
    """A tensor of the right device and layout without storage (a subclass that wraps others, a
    fake tensor) is refused, not taken for a gradient that is left out."""
    numels, dtypes = (ctypes.c_int64 * 1)(8), (ctypes.c_int32 * 1)(1)
    class Wrapper(torch.Tensor):
        @classmethod
        def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
            raise AssertionError("no operation is expected")

    make = lambda n: torch.Tensor._make_wrapper_subclass(  # noqa: E731
        Wrapper, (n,), dtype=torch.float32, device="cuda:0")
    with FakeTensorMode():
        fake = torch.empty(8, device="cuda:0")
    for t in (make(8), fake):
        assert t.is_cuda and t.is_contiguous()
        assert L.tensor_addresses([t], numels, dtypes, 0) == 0
    assert list(L.tensor_addresses([make(0)], (ctypes.c_int64 * 1)(0), dtypes, 0)) == [None]


def test_entries_at():
    at = L.args().entries_at
    a, b, c = torch.zeros(4), torch.zeros(2), torch.zeros(0)
    dicts, keys = [{"x": a, "n": 3}, {"x": b, "y": c}], ("x", "y")
    want = (ctypes.c_uint64 * 4)(a.data_ptr(), 0, b.data_ptr(), 0)
    assert at(dicts, keys, want) and at([], keys, (ctypes.c_uint64 * 0)())
    for i, k, v in ((0, "x", a.clone()), (0, "y", b), (1, "x", a), (1, "x", None), (1, "y", a)):
        other = [dict(d) for d in dicts]
        other[i][k] = v
        assert not at(other, keys, want)
    assert at([{"x": a, "y": "text"}, {"x": b}], keys, want) and not at([{}, None], keys, want)
    with FakeTensorMode():
        fake = torch.empty(8)
    assert not at([{"x": fake}], ("x",), (ctypes.c_uint64 * 1)(a.data_ptr()))
    for args in ((dicts, keys, (ctypes.c_uint64 * 3)()), (dicts, keys[:1], want)):
        with pytest.raises(ValueError):
            at(*args)
    with pytest.raises(TypeError):
        at(tuple(dicts), keys, want)
    with pytest.raises(TypeError):
        at([{}], ([],), (ctypes.c_uint64 * 1)())                        # an unhashable key


@pytest.mark.parametrize("small,change,error", [
    (False, {}, ValueError),                                            # CPU tensors
    (False, dict(exp_avgs=[]), ValueError),
    (False, dict(exp_avgs=[torch.zeros(301)]), ValueError),
    (False, dict(params=[torch.zeros(600)[::2]]), ValueError),
    (False, dict(exp_avgs=[torch.zeros(300, dtype=torch.bfloat16)]), TypeError),
    (False, dict(params=[torch.zeros(300, dtype=torch.float16)]), TypeError),
    (False, dict(grad_dtypes=[torch.float64]), TypeError),
    (False, dict(masters=[torch.zeros(300, dtype=torch.bfloat16)]), TypeError),
    (False, dict(wd_muls=[1.0, 2.0]), ValueError),
    (True, {}, ValueError),
    (True, dict(exp_avg_scales=None), ValueError),
    (True, dict(exp_avg_scales=[torch.zeros(2, dtype=torch.uint8)]), TypeError),
    (True, dict(exp_avg_scales=[torch.zeros(3, dtype=torch.uint8).view(torch.float8_e8m0fnu)]),
     ValueError),
    (True, dict(exp_avg_sqs=[torch.zeros(300)]), TypeError),
], ids=str)
def test_adamw_plan_refuses(small, change, error):
    with pytest.raises(error):
        om.AdamWPlan(**{**cpu_args(small=small), **change})


def test_cpu_tensors_are_refused_not_stepped():
    p = torch.nn.Parameter(torch.ones(5))
    p.grad = torch.ones(5)
    for fn in (lambda: om.grad_norm([p.grad]), lambda: om.clip_grad_norm_([p], 1.0),
               lambda: om.AdamW([p]).step(), lambda: om.AdamW([p], state_bits=8).step()):
        with pytest.raises(ValueError):
            fn()
    assert torch.equal(p.detach(), torch.ones(5)) and torch.equal(p.grad, torch.ones(5))


def test_optimizer_options():
    p = [torch.nn.Parameter(torch.ones(5)) for _ in range(2)]
    with pytest.raises(ValueError):
        om.AdamW(p, state_bits=16)
    opt = om.AdamW([{"params": p[:1], "state_bits": 8}, {"params": p[1:], "wd_mul": 0.0}],
                   max_grad_norm=1.0, seed=5)
    assert [g["state_bits"] for g in opt.param_groups] == [8, 32]
    with pytest.raises(ValueError):
        opt.add_param_group({"params": [torch.nn.Parameter(torch.ones(2))], "state_bits": 4})
    assert len(opt.param_groups) == 2
    opt.step()                                    # no gradients: nothing to do
    assert opt.last_grad_norm is None


def test_state_dict_keeps_the_states_dtypes():
    def make():
        p = [torch.nn.Parameter(torch.randn(300).to(torch.bfloat16)) for _ in range(2)]
        opt = om.AdamW([{"params": p[:1], "state_bits": 8}, {"params": p[1:]}], master_weights=True)
        for g in opt.param_groups:
            opt._init_state(g["params"][0], g)
        return p, opt
    p, opt = make()
    for st in opt.state.values():
        st["step"] = 7
        for k, v in st.items():
            if torch.is_tensor(v):
                raw = v.view(torch.uint8)
                raw.copy_(torch.randint(0, 100, raw.shape, dtype=torch.uint8))
    _, other = make()
    other.load_state_dict(opt.state_dict())
    for a, b in zip(opt.state.values(), other.state.values()):
        assert b["step"] == 7 and a.keys() == b.keys()
        for k, v in a.items():
            if torch.is_tensor(v):
                assert b[k].dtype == v.dtype and b[k].data_ptr() != v.data_ptr()
                assert torch.equal(b[k].view(torch.uint8), v.view(torch.uint8))
    assert opt.state[p[0]]["exp_avg"].dtype == torch.float8_e4m3fn
    assert opt.state[p[1]]["exp_avg"].dtype == opt.state[p[0]]["master"].dtype == torch.float32


def test_state_dict_of_torch_adamw_loads():
    p = torch.nn.Parameter(torch.randn(7))
    theirs = torch.optim.AdamW([p], lr=3e-4, weight_decay=0.2)
    p.grad = torch.randn(7)
    theirs.step()
    theirs.step()
    mine = om.AdamW([p])
    mine.load_state_dict(theirs.state_dict())
    g, st = mine.param_groups[0], mine.state[p]
    assert g["lr"] == 3e-4 and g["weight_decay"] == 0.2 and g["state_bits"] == 32 and g["wd_mul"] == 1.0
    assert st["step"] == 2 and type(st["step"]) is int
    assert torch.equal(st["exp_avg"], theirs.state[p]["exp_avg"])


@pytest.mark.parametrize("make", [
    lambda p: torch.optim.AdamW(p, amsgrad=True), lambda p: torch.optim.AdamW(p, maximize=True),
    lambda p: torch.optim.Adam(p, weight_decay=0.1)], ids=["amsgrad", "maximize", "coupled"])
def test_state_dict_of_another_step_is_refused(make):
    p = torch.nn.Parameter(torch.ones(5))
    opt = om.AdamW([p], lr=0.5)
    with pytest.raises(ValueError):
        opt.load_state_dict(make([p]).state_dict())
    assert opt.param_groups[0]["lr"] == 0.5 and not opt.state
    opt.load_state_dict(torch.optim.Adam([p], lr=0.25).state_dict())      # nothing decays
    assert opt.param_groups[0]["lr"] == 0.25


def test_optimizer_copies_and_checkpoints():
    import copy
    import io
    p = torch.nn.Parameter(torch.randn(300))
    opt = om.AdamW([p], state_bits=8, max_grad_norm=2.0, skip_nonfinite=True)
    opt._init_state(p, opt.param_groups[0])
    opt.state[p]["exp_avg"].view(torch.uint8).fill_(0x31)
    other = copy.deepcopy(opt)
    q = other.param_groups[0]["params"][0]
    assert other.max_grad_norm == 2.0 and other.skip_nonfinite and other._plans == {}
    assert other.state[q]["exp_avg"].dtype == torch.float8_e4m3fn
    other.step()                                  # no gradients: nothing to do
    file = io.BytesIO()
    torch.save(opt.state_dict(), file)
    file.seek(0)
    other.load_state_dict(torch.load(file, weights_only=True))
    for k, v in opt.state[p].items():
        if torch.is_tensor(v):
            assert other.state[q][k].dtype == v.dtype
            assert torch.equal(other.state[q][k].view(torch.uint8), v.view(torch.uint8))


def test_c_program_uses_the_abi(tmp_path):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    exe = tmp_path / "adamw_check"
    pkg = os.path.dirname(L.LIB_PATH)
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic",
                    "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(root, "include"), "-isystem",
                    os.path.join(rocm, "include"), os.path.join(root, "tests", "c_abi", "adamw_check.c"),
                    "-o", str(exe), "-L", pkg, "-lmuon", f"-Wl,-rpath,{pkg}",
                    f"-Wl,-rpath,{rocm}/lib", "-L", f"{rocm}/lib", "-lamdhip64"], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "abi ok" in r.stdout, r.stdout + r.stderr


def torch_state_dict(ps, steps=2, **kw):
    """The state dict of a torch.optim.AdamW after steps with random gradients."""
    theirs = torch.optim.AdamW(ps, **kw)
    for _ in range(steps):
        for p in ps:
            p.grad = torch.randn_like(p)
        theirs.step()
    for p in ps:
        p.grad = None
    return theirs.state_dict()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32, torch.float64], ids=str)
def test_moments_of_torch_adamw_become_float32(dt):
    """torch's moments have the dtype of the parameters that they were saved beside."""
    p = [torch.nn.Parameter(torch.randn(s).to(dt)) for s in ((300,), (3, 5))]
    saved = torch_state_dict(p)
    q = [torch.nn.Parameter(x.detach().to(torch.bfloat16)) for x in p]
    mine = om.AdamW(q)
    mine.load_state_dict(saved)
    for i, x in enumerate(q):
        st = mine.state[x]
        assert st["step"] == 2 and "exp_avg_scale" not in st
        for k in ("exp_avg", "exp_avg_sq"):
            assert saved["state"][i][k].dtype == dt and st[k].dtype == torch.float32
            assert st[k].shape == x.shape and torch.equal(st[k], saved["state"][i][k].float())


def test_moments_of_torch_adamw_become_8_bit_states():
    """As adamw.h defines them, by the oracle: m and sqrt(v) to nearest, v = 0 only where it was;
    and at the ends of fp32's range."""
    import numpy as np
    import oracle.adamw as oa
    r = np.random.default_rng(0)
    for n in (1, 255, 256, 2500):
        p = torch.nn.Parameter(torch.zeros(n))
        saved = torch_state_dict([p])
        m = torch.tensor(r.normal(0, 1, n) * 10.0 ** r.uniform(-40, 3, n), dtype=torch.float32)
        v = torch.tensor(10.0 ** r.uniform(-44, 4, n), dtype=torch.float32)
        if n > 1000:
            v[1::3] = 0.0
            top = torch.finfo(torch.float32).max
            m[300], m[301], v[600], v[1200] = top, -top, top, math.inf
            m[900], m[1500], v[1600] = math.nan, -math.inf, math.nan
            m[1800:2050], v[2060:] = 0.0, 0.0                         # whole blocks among them
            m[2100:2300] = 1e-42
        saved["state"][0].update(exp_avg=m, exp_avg_sq=v)
        mine = om.AdamW([p], state_bits=8)
        saved["param_groups"][0]["state_bits"] = 8
        mine.load_state_dict(saved)
        st = mine.state[p]
        m, v = m.double().numpy(), v.double().numpy()
        lost_m, lost_v = ~np.isfinite(m), np.isnan(v)
        m = np.where(np.isinf(m), np.sign(m) * float(torch.finfo(torch.float32).max), np.nan_to_num(m))
        v = np.nan_to_num(v, posinf=float(torch.finfo(torch.float32).max))
        root = np.sqrt(v.astype(np.float32)).astype(np.float64)
        for k, want, lost, floor in (("exp_avg", m, lost_m, False), ("exp_avg_sq", root, lost_v, True)):
            codes, scales = oa.hold(want, floor=floor)
            assert st[k].dtype == torch.float8_e4m3fn and st[k].shape == p.shape
            got = st[k].float().double().numpy()
            assert np.array_equal(np.isnan(got), lost)
            assert np.array_equal(got[~lost], codes.reshape(-1)[:n][~lost])
            assert np.array_equal(st[k + "_scale"].float().double().numpy(), scales)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=str)
def test_states_of_torch_adamw_get_masters(dt):
    """Without them the steps would round bf16 parameters each time, whatever the option says."""
    p = [torch.nn.Parameter(torch.randn(s).to(dt)) for s in (300, 7)]
    saved = torch_state_dict(p)
    q = [torch.nn.Parameter(p[0].detach().to(torch.bfloat16)), torch.nn.Parameter(p[1].detach().float())]
    mine = om.AdamW(q, master_weights=True)
    mine.load_state_dict(saved)
    master = mine.state[q[0]]["master"]
    assert master.dtype == torch.float32 and torch.equal(master, q[0].detach().float())
    assert "master" not in mine.state[q[1]]                   # an fp32 parameter needs none
    master.fill_(9.0)                                         # one that was saved is kept
    other = om.AdamW([torch.nn.Parameter(x.detach().clone()) for x in q], master_weights=True)
    other.load_state_dict(mine.state_dict())
    assert bool((other.state[other.param_groups[0]["params"][0]]["master"] == 9.0).all())
    plain = om.AdamW(q)
    plain.load_state_dict(saved)
    assert all("master" not in st for st in plain.state.values())


def test_groups_keep_the_options_that_torch_adamw_has_not():
    """Saved options are loaded; wd_mul, state_bits and the like stay as each group was built."""
    p = [torch.nn.Parameter(torch.randn(300)) for _ in range(3)]
    theirs = torch.optim.AdamW([{"params": p[:1]}, {"params": p[1:], "lr": 5e-4}], lr=2e-4, weight_decay=0.3)
    for x in p:
        x.grad = torch.randn_like(x)
    theirs.step()
    saved = theirs.state_dict()
    q = [torch.nn.Parameter(x.detach().to(torch.bfloat16)) for x in p]
    mine = om.AdamW([{"params": q[:1], "wd_mul": 0.0, "state_bits": 8, "seed": 9, "stochastic": False},
                     {"params": q[1:], "wd_mul": 2.0, "master_weights": False}],
                    master_weights=True, seed=4, weight_decay=0.01)
    mine.load_state_dict(saved)
    a, b = mine.param_groups
    own = ("wd_mul", "state_bits", "master_weights", "stochastic", "seed")
    assert [a[k] for k in own] == [0.0, 8, True, False, 9]
    assert [b[k] for k in own] == [2.0, 32, False, True, 4]
    assert (a["lr"], a["weight_decay"], b["lr"], b["weight_decay"]) == (2e-4, 0.3, 5e-4, 0.3)
    assert mine.state[q[0]]["exp_avg"].dtype == torch.float8_e4m3fn and "master" in mine.state[q[0]]
    assert mine.state[q[1]]["exp_avg"].dtype == torch.float32 and "master" not in mine.state[q[1]]
    other = om.AdamW([{"params": q[:1]}, {"params": q[1:]}])        # its own dict brings them all
    other.load_state_dict(mine.state_dict())
    assert [[g[k] for k in own] for g in other.param_groups] == [[g[k] for k in own] for g in (a, b)]


@pytest.mark.parametrize("bits", [32, 8])
def test_a_state_is_made_whole_or_not_at_all(bits, monkeypatch):
    """Memory that runs out in the middle leaves nothing behind that a later step would take for
    a state."""
    p = torch.nn.Parameter(torch.randn(300).to(torch.bfloat16))
    opt = om.AdamW([p], state_bits=bits, master_weights=True)
    zeros, calls = torch.zeros, []

    def short(*args, **kw):
        calls.append(args)
        if len(calls) == 2:
            raise torch.OutOfMemoryError("out of memory")
        return zeros(*args, **kw)

    monkeypatch.setattr(torch, "zeros", short)
    with pytest.raises(torch.OutOfMemoryError):
        opt._init_state(p, opt.param_groups[0])
    assert not opt.state.get(p)
    opt._init_state(p, opt.param_groups[0])
    assert opt.state[p]["step"] == 0 and "master" in opt.state[p] and "exp_avg_sq" in opt.state[p]


@pytest.mark.parametrize("bad", [
    dict(lr=-1.0), dict(lr=math.nan), dict(lr=math.inf), dict(betas=(0.9, 1.5)), dict(betas=(-0.1, 0.9)),
    dict(betas=(0.9, 1 - 1e-9)), dict(betas=(0.9,)), dict(betas=(math.nan, 0.9)), dict(eps=-1.0),
    dict(eps=math.inf), dict(weight_decay=-0.1), dict(weight_decay=1e39), dict(wd_mul=math.nan),
    dict(wd_mul=3e38, weight_decay=10.0)], ids=str)
def test_options_are_checked_where_they_are_given(bad):
    """...and not by the first step."""
    p = [torch.nn.Parameter(torch.ones(5)) for _ in range(2)]
    with pytest.raises(ValueError):
        om.AdamW(p, **bad)
    opt = om.AdamW(p[:1])
    with pytest.raises(ValueError):
        opt.add_param_group({"params": p[1:], **bad})
    assert len(opt.param_groups) == 1
    opt.add_param_group({"params": p[1:], "lr": 0.0, "betas": (0.0, 0.0), "eps": 0.0, "weight_decay": 0.0})


@pytest.mark.parametrize("bad", [-1.0, math.nan])
def test_max_grad_norm_is_checked_where_it_is_given(bad):
    with pytest.raises(ValueError):
        om.AdamW([torch.nn.Parameter(torch.ones(5))], max_grad_norm=bad)
    om.AdamW([torch.nn.Parameter(torch.ones(5))], max_grad_norm=0.0)


@pytest.mark.parametrize("bad", [dict(betas=0.9), dict(lr="fast"), dict(wd_mul=1e39, weight_decay=1e-9)], ids=str)
def test_a_refused_group_is_not_kept(bad):
    """Also where an option is not a number at all, or fits fp32 only in the product."""
    p = [torch.nn.Parameter(torch.ones(5)) for _ in range(2)]
    opt = om.AdamW(p[:1])
    with pytest.raises((TypeError, ValueError)):
        opt.add_param_group({"params": p[1:], **bad})
    assert len(opt.param_groups) == 1


@no_gpu_only
def test_check_returns_what_the_step_would():
    ents = entries()
    ents[2]["wd"] = 3e38
    plan = create(ents)
    cfg, other = L.muon_adamw_config_default(), L.muon_adamw_config_default()
    other.step = 0
    free, P = BASE + (64 << 20), L.make_pointers
    for grads, n, c in ((P([None] * 3), 3, other), (P([None] * 3), 2, cfg), (None, 3, cfg),
                        (P([free + 2, None, None]), 3, cfg), (P([BASE, None, None]), 3, cfg),
                        (P([free, None, None]), 3, cfg)):                     # no table yet
        want = status_of(L.muon_adamw_step, plan, grads, n, c, 0)
        assert status_of(L.muon_adamw_check, plan, grads, n, c) == want
    assert status_of(L.muon_adamw_check, None, P([None] * 3), 3, cfg)[0] == INV
    assert L.lib().muon_adamw_check(plan, P([None] * 3), 3, None) == INV
    cfg.weight_decay = 10.0
    assert status_of(L.muon_adamw_check, plan, P([None] * 3), 3, cfg)[0] == INV
    cfg.weight_decay = 0.0
    L.muon_adamw_check(plan, P([None] * 3), 3, cfg)
    L.muon_adamw_plan_destroy(plan)


def test_states_of_another_optimizer_load_as_they_are():
    """torch's Adamax has a first moment and no second one."""
    p = torch.nn.Parameter(torch.randn(7))
    theirs = torch.optim.Adamax([p])
    p.grad = torch.randn(7)
    theirs.step()
    mine = om.AdamW([p], master_weights=True)
    mine.load_state_dict(theirs.state_dict())
    assert torch.equal(mine.state[p]["exp_avg"], theirs.state[p]["exp_avg"])
    assert "exp_avg_sq" not in mine.state[p] and "master" not in mine.state[p]
