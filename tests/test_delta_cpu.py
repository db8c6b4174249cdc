"""The delta-rule and norm entry points without a GPU: struct layouts, refusals on the host, the
workspace query, the Python binding's checks, and the kernels' registers."""

from __future__ import annotations

import ctypes
import re
import struct
import subprocess
import sys
from pathlib import Path

import pytest
import torch

ROOT = Path(__file__).resolve().parents[1]
BASE = 1 << 30  # an address that is only looked at


@pytest.fixture(scope="module")
def ssu():
    from selective_state_update_02_gb300 import _build
    _build.build()
    import selective_state_update_02_gb300 as m
    m.lib()
    return m


@pytest.fixture()
def handle():
    """Zeros but for the number of SMs (struct ssu_handle_s): enough for calls that are refused."""
    return ctypes.create_string_buffer(struct.pack("ii", 0, 152), 4096)


def test_struct_layouts(ssu, tmp_path):
    names = ["ssu_delta_strides_t", "ssu_norm_args_t"]
    lines = []
    for s in names:
        lines += [f'printf("{s} {f} %zu %zu\\n", offsetof({s}, {f}), sizeof((({s} *)0)->{f}));'
                  for f, *_ in getattr(ssu, s)._fields_]
        lines.append(f'printf("{s} end %zu 0\\n", sizeof({s}));')
    (tmp_path / "layout.c").write_text(
        '#include <stddef.h>\n#include <stdio.h>\n#include "ssu.h"\nint main(void) {\n' +
        "\n".join(lines) + "\nreturn 0;\n}\n")
    subprocess.run(["gcc", "-std=c99", "-I", str(ROOT / "include"), str(tmp_path / "layout.c"),
                    "-o", str(tmp_path / "layout")], check=True)
    out = subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True)
    end = 0
    for line in out.stdout.splitlines():
        s, field, offset, size = line.split()
        cls = getattr(ssu, s)
        assert int(offset) == end, (s, field)  # no bytes between the fields
        if field == "end":
            assert ctypes.sizeof(cls) == int(offset)
            end = 0
        else:
            f = getattr(cls, field)
            assert (f.offset, f.size) == (int(offset), int(size)), (s, field)
            end += int(size)


def delta_call(ssu, handle, prompts, shape=(), strides=(), ptrs=(), scale=1.0, eps=1e-6, tokens=70,
               workspace=(BASE, 1 << 40)):
    """Status of a call with addresses that nothing reads: what is not refused ends at the missing
    device."""
    sizes = dict(batch=2, nheads=4, headdim=64, dstate=128, ngroups=2, pool_size=4, index_dtype=0,
                 state_dtype=0)
    sizes.update(shape)
    s = ssu.ssu_shape_t(*sizes.values())
    st = ssu.ssu_delta_strides_t()
    values = dict(state=(4 * 64 * 128, 64 * 128, 128), q=(256, 128), k=(256, 128), v=(256, 64),
                  out=(256, 64), dt=(4, 1), b=(4, 1), dt_bias=1, A=1, idx=1)
    values.update(strides)
    for k, v in values.items():
        if isinstance(v, tuple):
            getattr(st, k)[:] = v
        else:
            setattr(st, k, v)
    names = ["pool", "slots", *(("cu", "fresh") if prompts else ()), "q", "k", "v", "dt",
             "dt_bias", "A", "b", "out"]
    where = dict.fromkeys(names, BASE)
    where.update(ptrs)
    args = [ctypes.addressof(handle) if handle else None, *(where[n] for n in names),
            ctypes.byref(s), ctypes.byref(st)]
    if prompts:
        return ssu.lib().ssu_delta_prompts(*args, tokens, scale, eps, *workspace, None)
    return ssu.lib().ssu_delta_update(*args, scale, eps, None)


REFUSALS = [
    (1, dict(shape=dict(batch=-1))), (1, dict(shape=dict(ngroups=3))),
    (1, dict(shape=dict(index_dtype=2))), (1, dict(shape=dict(state_dtype=5))),
    (2, dict(shape=dict(dstate=96))), (2, dict(shape=dict(nheads=70000, ngroups=1))),
    (2, dict(shape=dict(headdim=2 ** 21))), (2, dict(shape=dict(batch=2 ** 30))),
    (1, dict(strides=dict(q=(-1, 128)))), (1, dict(strides=dict(idx=-1))),
    (1, dict(strides=dict(b=(4, -1)))), (3, dict(strides=dict(state=(4 * 64 * 128, 64 * 128, 130)))),
    (3, dict(shape=dict(state_dtype=1), strides=dict(state=(4 * 64 * 128, 64 * 128, 132)))),
    (3, dict(ptrs=dict(pool=BASE + 8))), (3, dict(ptrs=dict(slots=BASE + 2))),
    (3, dict(shape=dict(index_dtype=1), ptrs=dict(slots=BASE + 4))),
    (3, dict(ptrs=dict(k=BASE + 1))), (3, dict(ptrs=dict(A=BASE + 2))),
    *((1, dict(ptrs={k: None})) for k in ("pool", "slots", "q", "k", "v", "dt", "dt_bias", "A", "b",
                                          "out")),
    (1, dict(scale=float("nan"))), (1, dict(scale=float("inf"))), (1, dict(eps=float("nan"))),
]


@pytest.mark.parametrize("prompts", [False, True])
@pytest.mark.parametrize("status,change", REFUSALS, ids=str)
def test_delta_refusals(ssu, handle, prompts, status, change):
    assert delta_call(ssu, handle, prompts, **change) == status
    assert ssu.last_error()


@pytest.mark.parametrize("status,change", [
    (1, dict(tokens=-1)), (1, dict(tokens=2 ** 31)), (1, dict(ptrs=dict(cu=None))),
    (3, dict(ptrs=dict(cu=BASE + 2))), (1, dict(workspace=(None, 0))),
    (1, dict(workspace=(BASE, 100))), (3, dict(workspace=(BASE + 128, 1 << 40)))], ids=str)
def test_delta_prompt_refusals(ssu, handle, status, change):
    assert delta_call(ssu, handle, True, **change) == status


def test_calls_of_nothing_are_accepted(ssu, handle):
    none = dict.fromkeys(("pool", "slots", "q", "k", "v", "dt", "dt_bias", "A", "b", "out"))
    for prompts in (False, True):
        assert delta_call(ssu, handle, prompts, shape=dict(batch=0), ptrs=none) == ssu.SSU_OK
        assert delta_call(ssu, None, prompts) == ssu.SSU_ERR_INVALID_ARG


def query(ssu, handle, tokens=2000, **change):
    sizes = dict(batch=2, nheads=4, headdim=64, dstate=128, ngroups=2, pool_size=4, index_dtype=0,
                 state_dtype=0)
    sizes.update(change)
    n = ctypes.c_int64(-1)
    st = ssu.lib().ssu_delta_workspace_bytes(
        ctypes.addressof(handle), ctypes.byref(ssu.ssu_shape_t(*sizes.values())), tokens,
        ctypes.byref(n))
    return st, n.value


def test_workspace_query(ssu, handle):
    for status, change in ((1, dict(ngroups=0)), (1, dict(batch=-1)), (1, dict(tokens=-1)),
                           (1, dict(tokens=2 ** 31)), (2, dict(dstate=32)), (1, dict(index_dtype=3)),
                           (2, dict(batch=2 ** 30))):
        assert query(ssu, handle, **change) == (status, -1)
    status, n = query(ssu, handle)
    # a record of 26 KiB for every chunk of 64 tokens and head, and the lists
    assert status == 0 and n >= (2000 // 64 + 2) * 4 * 26 * 1024 and n % 256 == 0
    assert query(ssu, handle, dstate=256) == (0, 0)  # token by token
    assert query(ssu, handle, tokens=20) == (0, 0)
    assert query(ssu, handle, batch=0) == (0, 0)
    # past 32 GB of records a call runs token by token
    assert query(ssu, handle, tokens=2 ** 31 - 1) == (0, 0)
    assert query(ssu, handle, tokens=18_000_000)[1] > 2 ** 34


@pytest.mark.parametrize("status,change", [
    (1, dict(tokens=-1)), (1, dict(tokens=2 ** 31)), (1, dict(out_dtype=2)),
    (1, dict(residual_dtype=2)), (2, dict(width=4)), (2, dict(width=516)), (2, dict(width=32776)),
    (2, dict(group=48)), (2, dict(group=0)), (2, dict(group=1024)), (2, dict(width=520)),
    (1, dict(eps=-1.0)), (1, dict(eps=float("nan"))), (1, dict(x=-8)), (3, dict(x=513)),
    (3, dict(residual=BASE + 4)), (3, dict(out=BASE + 4)), (3, dict(weight=BASE + 4)),
    (3, dict(scales=BASE + 2)), (1, dict(weight=None)), (1, dict(scales=None)),
    (1, dict(scales_=(0, 1))), (1, dict(scales_=(4, 0))), (1, dict(scales_=(-4, 1))),
    (1, dict(out_=504)), (1, dict(residual_=504)), (3, dict(out_=516)),
    (3, dict(out_dtype=0, out=BASE + 8))], ids=str)
def test_norm_refusals(ssu, handle, status, change):
    # (names with an underscore: the strides, where the pointer has the same name)
    strides = {k[:-1]: v for k, v in change.items() if k.endswith("_")}
    change = {k: v for k, v in change.items() if not k.endswith("_")}
    pointers = {k: change[k] for k in ("residual", "scales", "weight", "out") if k in change}
    fields = {k: v for k, v in change.items() if k not in pointers} | strides
    args = ssu.ssu_norm_args_t(tokens=5, width=512, group=128, residual_dtype=0, out_dtype=1, x=512,
                               residual=512, out=512)
    args.scales[:] = (4, 1)
    eps = fields.pop("eps", 1e-6)
    for k, v in fields.items():
        if k == "scales":
            args.scales[:] = v
        else:
            setattr(args, k, v)
    where = dict(x=BASE, residual=BASE, weight=BASE, out=BASE, scales=BASE)
    where.update(pointers)
    got = ssu.lib().ssu_add_norm(ctypes.addressof(handle), where["x"], where["residual"],
                                 where["weight"], where["out"], where["scales"],
                                 ctypes.byref(args), eps, None)
    assert got == status and ssu.last_error()


def test_norm_of_no_tokens_and_without_a_handle(ssu, handle):
    a = ssu.ssu_norm_args_t(tokens=0, width=64)
    f = ssu.lib().ssu_add_norm
    assert f(ctypes.addressof(handle), None, None, None, None, None, ctypes.byref(a), 1e-6,
             None) == ssu.SSU_OK
    assert f(None, None, None, None, None, None, ctypes.byref(a), 1e-6,
             None) == ssu.SSU_ERR_INVALID_ARG
    assert f(ctypes.addressof(handle), None, None, None, None, None, None, 1e-6,
             None) == ssu.SSU_ERR_INVALID_ARG


def delta_tensors(T=20, H=2, P=64, N=128, G=1):
    bf = torch.bfloat16
    return dict(pool=torch.zeros(4, H, P, N), slots=torch.zeros(1, dtype=torch.int32),
                cu=torch.tensor([0, T], dtype=torch.int32), q=torch.zeros(T, G, N, dtype=bf),
                k=torch.zeros(T, G, N, dtype=bf), v=torch.zeros(T, H, P, dtype=bf),
                dt=torch.zeros(T, H, dtype=bf), dt_bias=torch.zeros(H), A=torch.zeros(H),
                b=torch.zeros(T, H, dtype=bf), out=torch.zeros(T, H, P, dtype=bf))


@pytest.mark.parametrize("error,change", [
    (TypeError, dict(q=torch.zeros(20, 1, 128))), (TypeError, dict(cu=torch.zeros(2).long())),
    (TypeError, dict(v=None)), (TypeError, dict(dt=torch.zeros(20, 2))),
    (TypeError, dict(pool=torch.zeros(4, 2, 64, 128).half())),
    (ValueError, dict(cu=torch.zeros(3, dtype=torch.int32))),
    (ValueError, dict(k=torch.zeros(20, 2, 128).bfloat16())),
    (ValueError, dict(b=torch.zeros(19, 2).bfloat16())),
    (ValueError, dict(out=torch.zeros(20, 2, 63).bfloat16())),
    (ValueError, dict(q=torch.zeros(20, 128, 1).bfloat16().transpose(1, 2))),
    (ValueError, {})], ids=str)  # host tensors
def test_binding_refusals(ssu, error, change):
    args = {**delta_tensors(), **change}
    with pytest.raises(error):
        ssu.ssu_delta_prompts(0, *args.values(), stream=0)
    if "cu" in change:
        return
    args.pop("cu")
    with pytest.raises(error):
        ssu.ssu_delta_update(0, *args.values(), stream=0)


def test_norm_binding_refusals(ssu):
    x, w, out = torch.zeros(3, 64).bfloat16(), torch.ones(64), torch.zeros(3, 64).bfloat16()
    e4m3, scales = out.to(torch.float8_e4m3fn), torch.zeros(3, 2)
    for error, args, kw in (
            (ValueError, (x, w, out), {}), (TypeError, (x.float(), w, out), {}),
            (TypeError, (x, w.bfloat16(), out), {}), (TypeError, (x, w, out.half()), {}),
            (ValueError, (x, w[:8], out), {}), (ValueError, (x, w, out[:2]), {}),
            (ValueError, (x, w, e4m3), {}), (ValueError, (x, w, out), dict(scales=scales)),
            (ValueError, (x, w, e4m3), dict(scales=scales[:, :0])),
            (ValueError, (x, w, e4m3), dict(scales=torch.zeros(3, 3))),
            (TypeError, (x, w, e4m3), dict(scales=scales.bfloat16())),
            (TypeError, (x, w, out), dict(residual=x.half())),
            (ValueError, (x, w, out), dict(residual=x[:1]))):
        with pytest.raises(error):
            ssu.ssu_add_norm(0, *args, stream=0, **kw)


CALLS = """
import sys
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
import selective_state_update_02_gb300 as ssu

bf, i32 = torch.bfloat16, torch.int32
with FakeTensorMode():
    f = lambda *s, d=bf: torch.empty(*s, dtype=d, device="cuda")
    w = lambda *s: f(*s, d=torch.float32)
    if sys.argv[1] == "norm":
        run, many = (lambda x: ssu.ssu_add_norm(0, x, w(64), f(3, 64), stream=0)), f(2, 3, 64)
    else:
        many = f(2, 20, 2, 64)
        rest = (f(20, 2), w(2), w(2), f(20, 2), f(20, 2, 64))
        if sys.argv[1] == "step":
            run = lambda v: ssu.ssu_delta_update(0, w(40, 2, 64, 128), f(20, d=i32), f(20, 1, 128),
                                                 f(20, 1, 128), v, *rest, stream=0)
        else:
            run = lambda v: ssu.ssu_delta_prompts(0, w(4, 2, 64, 128), f(1, d=i32), f(2, d=i32),
                                                  f(20, 1, 128), f(20, 1, 128), v, *rest, stream=0)
    for _ in range(5):
        try:
            torch.vmap(run)(many)
        except RuntimeError as e:
            print("refused", e)
        else:
            print("accepted")
"""


@pytest.mark.parametrize("which", ["step", "prompts", "norm"])
def test_tensors_without_storage(ssu, which):
    r = subprocess.run([sys.executable, "-c", CALLS, which], cwd=ROOT, capture_output=True,
                       text=True, timeout=120)
    assert r.returncode == 0, (r.returncode, r.stderr[-2000:])
    assert r.stdout.count("refused") == 5 and "data pointer" in r.stdout, r.stdout


# unit -> kernel -> (most registers, most spilled bytes).  Chunks: 384 threads with half a row of
# the state each, one CTA per SM; the first pass: four CTAs of 128 threads per SM; one token: what
# its state loads in flight take; norms: 16 warps of the largest rows per SM.
BUDGETS = {
    "ssu_delta.cu": {"ssu_delta_mma_kernel": (168, 64), "ssu_delta_prep_kernel": (128, 0),
                     "ssu_delta_step_kernel": (128, 0), "ssu_delta_seq_kernel": (168, 0),
                     "ssu_delta_plan_kernel": (64, 0)},
    "ssu_norm.cu": {"ssu_add_norm_kernel": (128, 96)},
}


@pytest.mark.parametrize("unit", sorted(BUDGETS))
def test_register_budgets(tmp_path, unit):
    from selective_state_update_02_gb300 import _build
    csrc = ROOT / "selective_state_update_02_gb300" / "csrc"
    out = subprocess.run(
        [_build.nvcc_path(), *_build.ARCH, "-O3", "-std=c++17", "-I", str(ROOT / "include"), "-I",
         str(csrc), "-Xptxas", "-v", "-cubin", "-c", str(csrc / unit), "-o",
         str(tmp_path / "unit.cubin")], capture_output=True, text=True, timeout=600,
        check=True).stderr
    seen = set()
    for block in out.split("ptxas info    : Compiling entry function '")[1:]:
        name = block.split("'")[0]
        used = int(re.search(r"Used (\d+) registers", block).group(1))
        spill = int(re.search(r"(\d+) bytes spill stores", block).group(1))
        for kernel, (most, spilled) in BUDGETS[unit].items():
            if kernel in name:
                seen.add(kernel)
                assert used <= most and spill <= spilled, (name, used, spill)
    assert seen == set(BUDGETS[unit])


LARGEST = dict(batch=512, tokens=65536, nheads=32)


@pytest.fixture()
def nowhere():
    """A handle on a device that no machine has: what is not refused ends there (status 4)."""
    return ctypes.create_string_buffer(struct.pack("ii", 1 << 20, 152), 4096)


@pytest.mark.parametrize("batch", [1, 2, 16, 33, 256, 511])
@pytest.mark.parametrize("tokens", [1, 36, 37, 64, 400, 1000, 4097, 65535])
@pytest.mark.parametrize("nheads", [4, 32])
def test_a_workspace_for_the_largest_call_serves_all(ssu, nowhere, batch, tokens, nheads):
    """The query's answer does not fall where prompts, tokens or heads grow, and no call of smaller
    sizes is refused with a buffer of that many bytes (status 4: it went on to the device)."""
    at = dict(batch=batch, tokens=tokens, nheads=nheads)
    status, need = query(ssu, nowhere, **at)
    assert status == 0
    for k in LARGEST:
        for more in (at[k] + 1, 2 * at[k], LARGEST[k]):
            larger = dict(at, **{k: more * 2 if k == "nheads" and more % 2 else more})
            assert query(ssu, nowhere, **larger)[1] >= need, larger
    shape = dict(batch=batch, nheads=nheads, headdim=128, pool_size=1024)
    assert delta_call(ssu, nowhere, True, shape=shape, tokens=tokens, workspace=(BASE, need)) == 4
    most = query(ssu, nowhere, **LARGEST)[1]
    assert delta_call(ssu, nowhere, True, shape=shape, tokens=tokens, workspace=(BASE, most)) == 4


@pytest.mark.parametrize("nheads,batch,tokens,status", [
    (32, 1, 24, 4), (32, 1, 36, 1), (32, 1, 64, 1), (32, 8, 48, 4), (32, 8, 96, 1), (32, 16, 64, 4),
    (32, 16, 192, 1), (32, 128, 512, 4), (32, 128, 1024, 1), (64, 1, 16, 4), (64, 1, 24, 1),
    (64, 1, 36, 1), (64, 2, 28, 1), (64, 8, 48, 4), (64, 8, 96, 1), (64, 32, 96, 4),
    (64, 32, 256, 1), (64, 128, 1024, 1)], ids=str)
def test_calls_token_by_token_need_no_workspace(ssu, nowhere, nheads, batch, tokens, status):
    """Heads of 128 x 128 on 152 SMs, at points where one form was measured to be the faster one however
    a call's tokens are spread (or where all but one each are one prompt's): where that is the
    token-by-token form (status 4: the call went on), no workspace is asked for."""
    shape = dict(batch=batch, nheads=nheads, headdim=128, pool_size=1024)
    got = delta_call(ssu, nowhere, True, shape=shape, tokens=tokens, workspace=(None, 0))
    assert got == status, ssu.last_error()


# unit -> pattern of a kernel's instantiations -> (most registers, most spilled bytes): what the
# kernels' times were measured at.  Norms of up to four vectors a thread keep two CTAs of 512
# threads to an SM, those into e4m3 with a residual at 36 spilled bytes; eight vectors (rows past
# 16384 columns) one CTA.
MEASURED = {
    "ssu_delta.cu": {r"ssu_delta_mma_kernel": (164, 0), r"ssu_delta_prep_kernel": (124, 0),
                     r"ssu_delta_step_kernelILi8ELi128Ef": (96, 0),
                     r"ssu_delta_step_kernelILi4ELi64E": (80, 0)},
    "ssu_norm.cu": {r"ssu_add_norm_kernelILi[124]E.*Lb0E": (64, 0),
                    r"ssu_add_norm_kernelILi[12]E.*Lb1E": (64, 0),
                    r"ssu_add_norm_kernelILi4E.*Lb1E": (64, 36),
                    r"ssu_add_norm_kernelILi8E": (128, 52)},
}


@pytest.mark.parametrize("unit", sorted(MEASURED))
def test_registers_as_measured(tmp_path, unit):
    from selective_state_update_02_gb300 import _build
    csrc = ROOT / "selective_state_update_02_gb300" / "csrc"
    out = subprocess.run(
        [_build.nvcc_path(), *_build.ARCH, "-O3", "-std=c++17", "-I", str(ROOT / "include"), "-I",
         str(csrc), "-Xptxas", "-v", "-cubin", "-c", str(csrc / unit), "-o",
         str(tmp_path / "unit.cubin")], capture_output=True, text=True, timeout=600,
        check=True).stderr
    seen = set()
    for block in out.split("ptxas info    : Compiling entry function '")[1:]:
        name = block.split("'")[0]
        used = int(re.search(r"Used (\d+) registers", block).group(1))
        spill = int(re.search(r"(\d+) bytes spill stores", block).group(1))
        for kernel, (most, spilled) in MEASURED[unit].items():
            if re.search(kernel, name):
                seen.add(kernel)
                assert used <= most and spill <= spilled, (name, used, spill)
    assert seen == set(MEASURED[unit])
