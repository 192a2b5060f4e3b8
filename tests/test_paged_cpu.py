"""CPU checks of the dense operators' entry points: plans, workspace sizes, refusals before anything is launched."""
import ctypes
import os
import shutil
import subprocess
import sys
import sysconfig
import types
import warnings

import pytest
import torch


@pytest.fixture(scope="module")
def mono():
    from learned_product_hash_proj_b200 import build
    build.build()
    from learned_product_hash_proj_b200 import mono as m
    return m


BASE = dict(Hq=8, Hkv=2, d=64, page=64, pages=10, layers=2, rows=4, width=3, tokens=100)


@pytest.mark.parametrize("change,status", [
    (dict(Hq=9), "MONO_ERR_INVALID"),                    # not a multiple of Hkv
    (dict(Hkv=0), "MONO_ERR_INVALID"),
    (dict(Hq=0), "MONO_ERR_INVALID"),
    (dict(page=0), "MONO_ERR_INVALID"),
    (dict(pages=0), "MONO_ERR_INVALID"),
    (dict(layers=0), "MONO_ERR_INVALID"),
    (dict(rows=-1), "MONO_ERR_INVALID"),
    (dict(width=-1), "MONO_ERR_INVALID"),
    (dict(tokens=-1), "MONO_ERR_INVALID"),
    (dict(scale=-0.5), "MONO_ERR_INVALID"),
    (dict(scale=float("nan")), "MONO_ERR_INVALID"),
    (dict(scale=float("inf")), "MONO_ERR_INVALID"),
    (dict(scale=1e35), "MONO_ERR_UNSUPPORTED"),          # beyond fp32 with its factors
    (dict(d=96), "MONO_ERR_UNSUPPORTED"),
    (dict(page=8), "MONO_ERR_UNSUPPORTED"),
    (dict(page=48), "MONO_ERR_UNSUPPORTED"),
    (dict(page=256), "MONO_ERR_UNSUPPORTED"),
    (dict(rows=20000), "MONO_ERR_UNSUPPORTED"),
    (dict(pages=1 << 25), "MONO_ERR_UNSUPPORTED"),       # pages*Hkv*page >= 2^31
    (dict(width=1 << 25), "MONO_ERR_UNSUPPORTED"),       # width*page >= 2^31
    (dict(rows=16384, width=1 << 20), "MONO_ERR_UNSUPPORTED"),
    (dict(tokens=(1 << 31) - 1), "MONO_ERR_UNSUPPORTED"),
    (dict(Hq=131072, Hkv=131072), "MONO_ERR_UNSUPPORTED"),
])
def test_plan_refusals(mono, change, status):
    with pytest.raises(mono.MonoError) as e:
        mono.PagedPlan(mono.PagedConfig(**{**BASE, **change}))
    assert mono.STATUS[e.value.status] == status


def test_unknown_dtype_is_refused(mono):
    with pytest.raises(ValueError, match="dtype"):
        mono.PagedPlan(mono.PagedConfig(**BASE, dtype="f16"))


@pytest.mark.parametrize("name", ["Hq", "Hkv", "d", "page", "pages", "layers", "rows", "width", "tokens"])
def test_sizes_beyond_32_bits_are_refused(mono, name):
    for v in (BASE[name] + (1 << 32), (1 << 31), -(1 << 31) - 1, 1 << 70):
        with pytest.raises(ValueError, match=name):
            mono.PagedPlan(mono.PagedConfig(**{**BASE, name: v}))


def test_plan_keeps_the_sizes_that_it_was_made_for(mono):
    # the checks of a call go by plan.cfg: a later change of the caller's object must not let other sizes through
    cfg = types.SimpleNamespace(**BASE, dtype="bf16", scale=0.0)
    plan = mono.PagedPlan(cfg)
    cfg.Hq, cfg.Hkv, cfg.width, cfg.layers, cfg.dtype = 2, 1, 1, 9, "f32"
    assert plan.cfg == mono.PagedConfig(**BASE) and plan.pool_shape == (2, 10, 2, 64, 64)
    with pytest.raises(ValueError, match="layer"):
        mono._layer(plan, 2)


def test_plans_and_workspace_sizes(mono):
    small = mono.PagedPlan(mono.PagedConfig(**BASE))
    assert small.workspace_bytes % 256 == 0 and small.pool_shape == (2, 10, 2, 64, 64)
    for more in (dict(rows=400), dict(pages=100000), dict(tokens=1 << 20)):
        assert mono.PagedPlan(mono.PagedConfig(**{**BASE, **more})).workspace_bytes > small.workspace_bytes
    for edge in (dict(rows=0), dict(width=0), dict(tokens=0), dict(scale=0.0), dict(page=16), dict(page=128)):
        assert mono.PagedPlan(mono.PagedConfig(**{**BASE, **edge})).workspace_bytes > 0
    ws = small.workspace("cpu")
    assert ws.numel() == small.workspace_bytes and (ws[:256] == 0).all()
    assert mono.lib().mono_paged_plan(None, None, None) == 3


def test_entry_points_refuse_before_launching(mono):
    lib = mono.lib()
    p = mono.PagedPlan(mono.PagedConfig(**BASE)).handle
    plan = mono.PagedPlan(mono.PagedConfig(**BASE))
    p = plan.handle
    f = ctypes.c_void_p(1 << 20)               # never dereferenced: validation fails first
    odd16 = ctypes.c_void_p((1 << 20) + 8)
    odd4 = ctypes.c_void_p((1 << 20) + 2)
    odd256 = ctypes.c_void_p((1 << 20) + 16)
    N = None
    # mono_prompt_attend(plan, n, total_q, total_k, Q, K, V, cu_q, cu_k, O, ws, stream)
    assert lib.mono_prompt_attend(N, 1, 5, 5, f, f, f, f, f, f, f, N) == 3
    assert lib.mono_prompt_attend(p, 1, 5, 5, f, f, f, f, f, f, N, N) == 4
    assert lib.mono_prompt_attend(p, 1, 5, 5, f, f, f, f, f, f, odd256, N) == 7
    assert lib.mono_prompt_attend(p, 5, 5, 5, f, f, f, f, f, f, f, N) == 1       # more sequences than rows
    assert lib.mono_prompt_attend(p, 1, 101, 5, f, f, f, f, f, f, f, N) == 1     # more tokens than the plan's
    assert lib.mono_prompt_attend(p, -1, 5, 5, f, f, f, f, f, f, f, N) == 1
    assert lib.mono_prompt_attend(p, 1, 5, -1, f, f, f, f, f, f, f, N) == 1
    assert lib.mono_prompt_attend(p, 1, 5, 5, N, f, f, f, f, f, f, N) == 3
    assert lib.mono_prompt_attend(p, 1, 5, 5, f, f, odd16, f, f, f, f, N) == 7
    assert lib.mono_prompt_attend(p, 1, 5, 5, f, f, f, odd4, f, f, f, N) == 7
    assert lib.mono_prompt_attend(p, 0, 5, 5, N, N, N, N, N, N, f, N) == 0       # nothing to do
    assert lib.mono_prompt_attend(p, 2, 0, 5, N, N, N, N, N, N, f, N) == 0
    # mono_paged_append(plan, layer, n, total, K, V, cu, table, lens, Kp, Vp, ws, stream)
    assert lib.mono_paged_append(p, 2, 1, 5, f, f, f, f, f, f, f, f, N) == 1     # layer
    assert lib.mono_paged_append(p, -1, 1, 5, f, f, f, f, f, f, f, f, N) == 1
    assert lib.mono_paged_append(p, 0, 5, 5, f, f, f, f, f, f, f, f, N) == 1
    assert lib.mono_paged_append(p, 0, 1, 5, f, f, f, N, f, f, f, f, N) == 3
    assert lib.mono_paged_append(p, 0, 1, 5, f, f, f, f, f, odd16, f, f, N) == 7
    assert lib.mono_paged_append(p, 0, 1, 0, N, N, N, N, N, N, N, f, N) == 0
    # mono_paged_attend(plan, layer, n, Q, table, lens, Kp, Vp, O, ws, stream)
    assert lib.mono_paged_attend(p, 0, 1, f, f, f, f, f, f, N, N) == 4
    assert lib.mono_paged_attend(p, 7, 1, f, f, f, f, f, f, f, N) == 1
    assert lib.mono_paged_attend(p, 0, 1, f, f, N, f, f, f, f, N) == 3
    assert lib.mono_paged_attend(p, 0, 1, odd16, f, f, f, f, f, f, N) == 7
    assert lib.mono_paged_attend(p, 0, 0, N, N, N, N, N, N, f, N) == 0
    # mono_paged_update(plan, n_in, table, lens, n_out, parents, grow, table_out, lens_out, Kp, Vp, ws, stream)
    g, h = ctypes.c_void_p(1 << 21), ctypes.c_void_p(1 << 22)
    assert lib.mono_paged_update(p, 1, f, f, 5, f, f, g, h, f, f, f, N) == 1
    assert lib.mono_paged_update(p, -1, f, f, 1, f, f, g, h, f, f, f, N) == 1
    assert lib.mono_paged_update(p, 1, f, f, 1, N, f, g, h, f, f, f, N) == 3
    assert lib.mono_paged_update(p, 1, f, g, 1, g, g, f, h, f, f, f, N) == 1     # table_out over table
    assert lib.mono_paged_update(p, 1, f, g, 1, g, g, h, g, f, f, f, N) == 1     # lens_out over lens
    assert lib.mono_paged_update(p, 1, f, g, 0, N, N, N, N, N, N, f, N) == 0
    # mono_paged_compact(plan, n, table, lens, table_out, Kp, Vp, ws, stream)
    assert lib.mono_paged_compact(p, 1, f, g, f, h, h, f, N) == 1                # in place
    assert lib.mono_paged_compact(p, 9, f, g, h, h, h, f, N) == 1
    assert lib.mono_paged_compact(p, 1, f, N, h, h, h, f, N) == 3
    assert lib.mono_paged_compact(p, 0, N, N, N, N, N, f, N) == 0
    st = mono.PagedStats()
    assert lib.mono_paged_stats(p, N, N, ctypes.byref(st)) == 4
    assert lib.mono_paged_stats(p, f, N, N) == 3


def test_outputs_over_inputs_and_calls_beyond_32_bits_are_refused(mono):
    lib = mono.lib()
    for dtype in ("bf16", "f32"):
        plan = mono.PagedPlan(mono.PagedConfig(**{**BASE, "dtype": dtype}))
        at = [ctypes.c_void_p((1 + i) << 24) for i in range(8)]     # never dereferenced: refused before any launch
        inside = ctypes.c_void_p((1 << 24) + 16)
        q, k, v, cu, ws = at[:5]
        for o in (q, inside, k, v):
            assert lib.mono_prompt_attend(plan.handle, 1, 5, 5, q, k, v, cu, cu, o, ws, None) == 1
        for o in (q, inside):
            assert lib.mono_paged_attend(plan.handle, 0, 1, q, cu, cu, k, v, o, ws, None) == 1
        wide = mono.PagedPlan(mono.PagedConfig(**{**BASE, "dtype": dtype, "Hq": 65535, "Hkv": 65535, "rows": 16384,
                                                  "tokens": 64, "page": 16}))
        far = ctypes.c_void_p(1 << 40)
        assert lib.mono_prompt_attend(wide.handle, 16384, 64, 5, q, k, v, cu, cu, far, ws, None) == 2


@pytest.mark.parametrize("call,written,read", [
    ("prompt", ["O", "ws"], ["Q", "K", "V", "cu_q", "cu_k"]),
    ("append", ["Kp", "Vp", "ws"], ["K", "V", "cu", "table", "lens"]),
    ("attend", ["O", "ws"], ["Q", "table", "lens", "Kp", "Vp"]),
    ("update", ["table_out", "lens_out", "Kp", "Vp", "ws"], ["table", "lens", "parents", "grow"]),
    ("compact", ["table_out", "Kp", "Vp", "ws"], ["table", "lens"]),
])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_what_is_written_overlaps_nothing(mono, dtype, call, written, read):
    # every pair, the two ranges starting together or one inside the other
    lib = mono.lib()
    cfg = {**BASE, "dtype": dtype, "pages": 9}
    plan = mono.PagedPlan(mono.PagedConfig(**cfg))
    p, es, n, t = plan.handle, 2 if dtype == "bf16" else 4, 3, 40
    pool = cfg["layers"] * cfg["pages"] * cfg["Hkv"] * cfg["page"] * cfg["d"] * es
    size = {"Q": (t if call == "prompt" else n) * 8 * 64 * es, "K": t * 2 * 64 * es, "cu_q": 4 * (n + 1), "lens": 4 * n,
            "table": 4 * n * cfg["width"], "Kp": pool, "ws": plan.workspace_bytes}
    size.update(O=size["Q"], V=size["K"], cu_k=size["cu_q"], cu=size["cu_q"], parents=size["lens"], grow=size["lens"],
                lens_out=size["lens"], table_out=size["table"], Vp=pool)
    run = {  # never dereferenced: refused before any launch
        "prompt": lambda a: lib.mono_prompt_attend(p, n, t, t, a["Q"], a["K"], a["V"], a["cu_q"], a["cu_k"], a["O"],
                                                   a["ws"], None),
        "append": lambda a: lib.mono_paged_append(p, 1, n, t, a["K"], a["V"], a["cu"], a["table"], a["lens"], a["Kp"],
                                                  a["Vp"], a["ws"], None),
        "attend": lambda a: lib.mono_paged_attend(p, 1, n, a["Q"], a["table"], a["lens"], a["Kp"], a["Vp"], a["O"],
                                                  a["ws"], None),
        "update": lambda a: lib.mono_paged_update(p, n, a["table"], a["lens"], n, a["parents"], a["grow"],
                                                  a["table_out"], a["lens_out"], a["Kp"], a["Vp"], a["ws"], None),
        "compact": lambda a: lib.mono_paged_compact(p, n, a["table"], a["lens"], a["table_out"], a["Kp"], a["Vp"],
                                                    a["ws"], None),
    }[call]
    apart = {name: (1 + i) << 28 for i, name in enumerate(written + read)}
    step = lambda name: 256 if name == "ws" else 16 if name in ("Q", "K", "V", "O", "Kp", "Vp") else 4
    pairs = [(w, x) for i, w in enumerate(written) for x in read + written[i + 1:]]
    for a, b in pairs + [(b, a) for a, b in pairs]:
        last = apart[a] + (size[a] - 1) // step(b) * step(b)      # the last place inside a where b may start
        for at in (apart[a], last):
            args = {k: ctypes.c_void_p(v) for k, v in {**apart, b: at}.items()}
            assert run(args) == 1, (a, b, at - apart[a])


def test_binding_refuses_host_tensors_and_wrong_shapes(mono):
    plan = mono.PagedPlan(mono.PagedConfig(**BASE))
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    kp, vp = plan.pools("cpu")
    ws = plan.workspace("cpu")
    with pytest.raises(ValueError, match="CUDA tensor"):
        mono.prompt_attend(plan, z(5, 8, 64), z(5, 2, 64), z(5, 2, 64), i(2), i(2), z(5, 512), ws)
    with pytest.raises(ValueError, match="CUDA tensor"):
        mono.paged_attend(plan, 0, z(2, 8, 64), i(2, 3), i(2), z(2, 512), kp, vp, ws)
    with pytest.raises(ValueError, match="CUDA tensor"):
        mono.paged_append(plan, 0, z(2, 2, 64), z(2, 2, 64), i(3), i(2, 3), i(2), kp, vp, ws)
    with pytest.raises(ValueError, match="CUDA tensor"):
        mono.paged_update(plan, i(2, 3), i(2), i(2), i(2), i(2, 3), i(2), kp, vp, ws)
    with pytest.raises(ValueError, match="CUDA tensor"):
        mono.paged_compact(plan, i(2, 3), i(2), i(2, 3), kp, vp, ws)
    with pytest.raises(ValueError, match="CUDA tensor"):
        mono.paged_stats(plan, ws)


def test_quick_way_declines_what_it_cannot_check(mono):
    # None and no exception: the checks in Python then say what is wrong
    from learned_product_hash_proj_b200 import _tensor_args as quick
    plan = mono.PagedPlan(mono.PagedConfig(**BASE))
    kp, vp = plan.pools("cpu")
    ws = plan.workspace("cpu")
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    good = [plan.quick, 0, torch.zeros(2, 8, 64, dtype=torch.bfloat16), i(2, 3), i(2),
            torch.zeros(2, 512, dtype=torch.bfloat16), kp, vp, ws, None]
    assert quick.paged_attend(*good) is None                       # not on a GPU
    for at in range(len(good)):
        for wrong in (None, 3, "x", [1], -1, 1 << 70):
            assert quick.paged_attend(*good[:at], wrong, *good[at + 1:]) is None
    for f, n in ((quick.prompt_attend, 9), (quick.paged_append, 11), (quick.paged_attend, 10), (quick.paged_update, 11),
                 (quick.paged_compact, 8)):
        for count in (0, 1, n - 1, n, n + 1):
            assert f(*([plan.quick] + [None] * n)[:count]) is None


# ---------------------------------------------------------------------------
# the quick way is optional
# ---------------------------------------------------------------------------
def package_copy(tmp_path, keep=lambda name: True):
    """The package in a place of its own: the built files that `keep` takes, the library as a link."""
    from learned_product_hash_proj_b200 import build
    to = tmp_path / "learned_product_hash_proj_b200"
    to.mkdir()
    for name in os.listdir(build.PKG):
        if name.endswith(".py") or (name.startswith("_tensor_args") and keep(name)):
            shutil.copy(os.path.join(build.PKG, name), to / name)
    os.symlink(build.LIB, to / "libmono.so")
    return tmp_path


USE = """
from learned_product_hash_proj_b200 import mono
import torch
plan = mono.PagedPlan(mono.PagedConfig(Hq=8, Hkv=2, d=64, rows=2, width=3))
i = lambda *s: torch.zeros(s, dtype=torch.int32)
z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
try:
    mono.paged_attend(plan, 0, z(2, 8, 64), i(2, 3), i(2), z(2, 512), *plan.pools("cpu"), plan.workspace("cpu"))
except ValueError as e:
    assert "CUDA tensor" in str(e)
    print("checked in Python")
"""


def run_python(code, at):
    return subprocess.run([sys.executable, "-c", code], cwd=at, env={**os.environ, "PYTHONPATH": str(at)},
                          capture_output=True, text=True, timeout=300)


def test_package_works_without_the_quick_way(mono, tmp_path):
    res = run_python(USE, package_copy(tmp_path, keep=lambda name: False))
    assert res.returncode == 0 and "checked in Python" in res.stdout, res.stderr


def test_package_works_with_a_torch_without_cuda(mono, tmp_path):
    # what such a torch lacks
    res = run_python("import torch\ndel torch._C._cuda_getDevice\n" + USE, package_copy(tmp_path))
    assert res.returncode == 0 and "checked in Python" in res.stdout, res.stderr


def test_package_works_with_another_exchange_table(mono, tmp_path):
    code = "import torch\ntorch.Tensor.__dlpack_c_exchange_api__ = object()\n"
    res = run_python(code + USE, package_copy(tmp_path))
    assert res.returncode == 0 and "checked in Python" in res.stdout, res.stderr


def test_build_goes_on_without_the_quick_way(mono, tmp_path, monkeypatch):
    from learned_product_hash_proj_b200 import build
    src = tmp_path / "wrong.cc"
    src.write_text("#include <no_such_header.h>\n")
    lib = tmp_path / "_tensor_args.so"
    lib.write_text("an earlier one")
    monkeypatch.setattr(build, "ARGS_SRC", str(src))
    monkeypatch.setattr(build, "ARGS_LIB", str(lib))
    monkeypatch.setattr(build, "ARGS_KEY", str(tmp_path / "key"))
    with pytest.warns(UserWarning, match="was not built"):
        assert build.build() == build.LIB
    assert not lib.exists()
    with warnings.catch_warnings():                                 # not tried again until something changes
        warnings.simplefilter("error")
        build.build()
    monkeypatch.setattr(build.importlib.metadata, "version", lambda name: "another")
    with pytest.warns(UserWarning, match="was not built"):
        build.build()


def test_quick_way_is_built_for_one_python_and_torch(mono, monkeypatch):
    from learned_product_hash_proj_b200 import build
    from learned_product_hash_proj_b200 import _tensor_args as quick
    assert os.path.samefile(quick.__file__, build.ARGS_LIB)
    assert build.ARGS_LIB.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    assert not os.path.exists(os.path.join(build.PKG, "_tensor_args.so"))
    assert not build._args_stale()
    monkeypatch.setattr(build.importlib.metadata, "version", lambda name: "another")
    assert build._args_stale()
