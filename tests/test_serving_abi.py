"""The serving entry points where no GPU is needed: the mirrored structures
against the C compiler's layout, workspaces, and what the C ABI and the Python
binding refuse before anything is launched."""
import ctypes
import os
import subprocess

import pytest

import lossless_entropy_coded_dfc_amd as dfc

torch = pytest.importorskip("torch")
U32, U64, I64, PTR, F32 = ctypes.c_uint32, ctypes.c_uint64, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float


class Cache(ctypes.Structure):
    _fields_ = [("k_dev", PTR), ("v_dev", PTR), ("k_stride", I64 * 3), ("v_stride", I64 * 3), ("n_pages", U32),
                ("page_size", U32), ("kv_heads", U32), ("head_dim", U32), ("dtype", U32)]


class Append(ctypes.Structure):
    _fields_ = [("cache", Cache), ("tokens", U64), ("k_dev", PTR), ("v_dev", PTR), ("k_src_stride", I64 * 2),
                ("v_src_stride", I64 * 2), ("slots", PTR), ("source_dtype", U32), ("q_heads", U32), ("q_dev", PTR),
                ("q_out_dev", PTR), ("q_stride", I64 * 2), ("q_out_stride", I64 * 2), ("rot_dim", U32),
                ("interleaved", U32), ("max_positions", U32), ("positions", PTR), ("rotary_dev", PTR),
                ("status_dev", PTR)]


class Norm(ctypes.Structure):
    _fields_ = [("q_norm_dev", PTR), ("k_norm_dev", PTR), ("dtype", U32), ("eps", F32)]


class Release(ctypes.Structure):
    _fields_ = [("n_requests", U32), ("max_pages", U32), ("page_size", U32), ("n_ring", U32), ("n_pages", U32),
                ("window", U32), ("sinks", U32), ("held_lens", PTR), ("keep_lens", PTR), ("block_table", PTR),
                ("table_stride", I64), ("free_pages", PTR), ("cursor", PTR), ("cursor_out", PTR), ("shared", PTR),
                ("workspace_dev", PTR), ("status_dev", PTR)]


class Fork(ctypes.Structure):
    _fields_ = [("n_requests", U32), ("max_pages", U32), ("page_size", U32), ("n_ring", U32), ("n_pages", U32),
                ("context_lens", PTR), ("parents", PTR), ("fork_lens", PTR), ("block_table", PTR),
                ("table_stride", I64), ("free_pages", PTR), ("cursor", PTR), ("cursor_out", PTR), ("shared", PTR),
                ("context_out", PTR), ("src", PTR), ("dst", PTR), ("status_dev", PTR)]


class Compact(ctypes.Structure):
    _fields_ = [("n_requests", U32), ("max_pages", U32), ("page_size", U32), ("n_ring", U32), ("n_pages", U32),
                ("context_lens", PTR), ("block_table", PTR), ("table_stride", I64), ("free_pages", PTR),
                ("cursor", PTR), ("shared", PTR), ("src", PTR), ("dst", PTR), ("used", PTR), ("workspace_dev", PTR),
                ("status_dev", PTR)]


class Verify(ctypes.Structure):
    _fields_ = [("n_requests", U32), ("vocab", U32), ("rows", U64), ("dtype", U32), ("logits_dev", PTR),
                ("logits_stride", I64), ("draft_logits_dev", PTR), ("draft_stride", I64), ("cu_rows", PTR),
                ("drafts", PTR), ("uniforms", PTR), ("temperature", PTR), ("accepted", PTR), ("tokens", PTR),
                ("workspace_dev", PTR), ("workspace_bytes", U64), ("status_dev", PTR)]


NAMES = [("dfc_append_args", Append), ("dfc_norm_args", Norm), ("dfc_release_args", Release), ("dfc_fork_args", Fork),
         ("dfc_compact_args", Compact), ("dfc_verify_args", Verify)]


@pytest.mark.parametrize("name,mirror", NAMES)
def test_layout(name, mirror, tmp_path):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    fields = [f[0] for f in mirror._fields_]
    lines = "\n".join(f'printf("%zu %zu\\n", offsetof({name}, {f}), sizeof(x.{f}));' for f in fields)
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text(f"#include <stddef.h>\n#include <stdio.h>\n#include \"dfc.h\"\n"
                   f"int main(void) {{ {name} x; (void)x; {lines}\n printf(\"%zu 0\\n\", sizeof(x)); return 0; }}\n")
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    got = [tuple(map(int, line.split())) for line in
           subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines()]
    assert got[-1][0] == ctypes.sizeof(mirror)
    assert got[:-1] == [(getattr(mirror, f).offset, getattr(mirror, f).size) for f in fields]


def refused(name, args, status, **changes):
    """What the C entry point answers with some fields changed (pointers are
    addresses that nothing reads before the refusal)."""
    a = type(args).from_buffer_copy(args)
    for k, v in changes.items():
        setattr(a, k, v)
    f = getattr(dfc.library(), name)
    f.argtypes = [ctypes.POINTER(type(a)), PTR]
    assert f(a, None) == status, changes


def test_release_refusals():
    good = Release(2, 4, 16, 8, 8, 0, 0, 256, 512, 1024, 4, 2048, 4096, 4112, 8192, 256, None)
    for change in (dict(page_size=0), dict(page_size=24), dict(n_ring=0), dict(n_pages=0), dict(n_pages=(1 << 30) + 1),
                   dict(held_lens=None), dict(keep_lens=None), dict(block_table=None), dict(table_stride=3),
                   dict(max_pages=0), dict(free_pages=None), dict(cursor=None), dict(cursor_out=None),
                   dict(cursor_out=4096), dict(shared=None), dict(workspace_dev=None), dict(workspace_dev=260),
                   dict(window=1 << 31), dict(sinks=1 << 31), dict(n_ring=1 << 31)):
        refused("dfc_paged_release", good, dfc.EINVAL, **change)
    refused("dfc_paged_release", good, dfc.EUNSUPPORTED, n_requests=65537)


def test_fork_refusals():
    good = Fork(2, 4, 16, 8, 8, 256, 512, None, 1024, 4, 2048, 4096, 4112, 8192, 768, 1280, 1536, None)
    for change in (dict(page_size=3), dict(n_ring=0), dict(n_pages=0), dict(context_lens=None), dict(parents=None),
                   dict(block_table=None), dict(table_stride=3), dict(free_pages=None), dict(cursor=None),
                   dict(cursor_out=None), dict(cursor_out=4096), dict(shared=None), dict(context_out=None),
                   dict(context_out=256), dict(context_out=512), dict(src=None), dict(dst=None), dict(src=256),
                   dict(dst=512), dict(dst=1280), dict(fork_lens=1536)):
        refused("dfc_paged_fork", good, dfc.EINVAL, **change)
    refused("dfc_paged_fork", good, dfc.EUNSUPPORTED, n_requests=65537)


def test_compact_refusals():
    good = Compact(2, 4, 16, 8, 8, 256, 1024, 4, 2048, 4096, 8192, 1280, 1536, 1792, 256, None)
    for change in (dict(page_size=3), dict(n_ring=0), dict(n_pages=0), dict(context_lens=None), dict(block_table=None),
                   dict(table_stride=3), dict(free_pages=None), dict(cursor=None), dict(shared=None), dict(src=None),
                   dict(dst=None), dict(dst=1280), dict(used=None), dict(workspace_dev=None), dict(workspace_dev=264)):
        refused("dfc_paged_compact", good, dfc.EINVAL, **change)
    refused("dfc_paged_compact", good, dfc.EUNSUPPORTED, n_requests=65537)


def test_copy_refusals():
    f = dfc.library().dfc_paged_copy
    f.argtypes = [ctypes.POINTER(Cache), U32, PTR, PTR, U32, PTR, PTR]
    s = (I64 * 3)(16 * 2 * 64, 2 * 64, 64)
    a, b = Cache(256, 512, s, s, 8, 16, 2, 64, 0), Cache(1024, 2048, s, s, 8, 16, 2, 64, 0)

    def call(*caches, src=256, dst=512, n=3):
        return f((Cache * len(caches))(*caches), len(caches), src, dst, n, None, None)

    assert call(a, b, n=0) == dfc.OK and f(None, 0, 256, 512, 3, None, None) == dfc.OK
    assert f(None, 1, 256, 512, 3, None, None) == dfc.EINVAL
    for src, dst in ((None, 512), (256, None), (256, 256)):
        assert call(a, b, src=src, dst=dst) == dfc.EINVAL
    for field, value in (("n_pages", 9), ("page_size", 8), ("kv_heads", 1), ("head_dim", 32), ("dtype", 1),
                         ("k_dev", None), ("v_dev", 520), ("head_dim", 60),
                         ("k_stride", (I64 * 3)(16 * 2 * 64, 64, 16 * 64))):
        c = Cache.from_buffer_copy(b)
        setattr(c, field, value)
        assert call(a, c) == dfc.EINVAL, field
    for field, value in (("dtype", 2), ("head_dim", 264), ("k_stride", (I64 * 3)(1 << 34, 64, 64))):
        c = Cache.from_buffer_copy(b)
        setattr(c, field, value)
        assert call(c) == dfc.EUNSUPPORTED, field


def test_norm_refusals():
    s = (I64 * 3)(16 * 2 * 64, 2 * 64, 64)
    rows = (I64 * 2)(128, 64)
    good = Append(Cache(256, 256, s, s, 8, 16, 2, 64, 0), 0, 256, 256, rows, rows, 256, 2, 2, 256, 512, rows, rows, 0, 0,
                  0, None, None, None)
    f = dfc.library().dfc_paged_append_normed
    f.argtypes = [ctypes.POINTER(Append), ctypes.POINTER(Norm), PTR]
    assert f(good, None, None) == dfc.OK and f(good, Norm(256, 256, 2, 1e-6), None) == dfc.OK
    for n in (Norm(260, 256, 2, 1e-6), Norm(256, 264, 2, 1e-6), Norm(256, None, 2, 0.0), Norm(256, None, 2, -1.0),
              Norm(256, None, 2, float("nan")), Norm(256, None, 2, float("inf"))):
        assert f(good, n, None) == dfc.EINVAL
    assert f(good, Norm(None, None, 9, 0.0), None) == dfc.OK  # nothing is normed
    for dtype in (1, 3):
        assert f(good, Norm(256, 256, dtype, 1e-6), None) == dfc.EUNSUPPORTED
    # in place only what is left as it is
    one = Append.from_buffer_copy(good)
    one.tokens, one.source_dtype, one.q_out_dev = 1, 0, 256
    assert f(one, Norm(256, None, 2, 1e-6), None) == dfc.EINVAL


def test_verify_refusals_and_workspace():
    good = Verify(2, 1000, 5, 2, 256, 1000, 512, 1000, 256, 256, 256, None, 256, 512, 256, 1 << 20, None)
    for change in (dict(cu_rows=None), dict(accepted=None), dict(tokens=None), dict(logits_dev=None), dict(drafts=None),
                   dict(uniforms=None), dict(workspace_dev=None), dict(workspace_dev=260), dict(logits_stride=999),
                   dict(draft_stride=999)):
        refused("dfc_verify_drafts", good, dfc.EINVAL, **change)
    for change in (dict(dtype=3), dict(vocab=0), dict(vocab=(1 << 30) + 1), dict(n_requests=65537), dict(rows=1 << 30)):
        refused("dfc_verify_drafts", good, dfc.EUNSUPPORTED, **change)
    lib = dfc.library()
    lib.dfc_verify_workspace.argtypes = [ctypes.POINTER(Verify), ctypes.POINTER(U64)]
    size = U64()
    assert lib.dfc_verify_workspace(good, ctypes.byref(size)) == dfc.OK and size.value > 0
    refused("dfc_verify_drafts", good, dfc.ESIZE, workspace_bytes=size.value - 1)
    both = size.value
    good.draft_logits_dev = None
    assert lib.dfc_verify_workspace(good, ctypes.byref(size)) == dfc.OK and size.value < both
    refused("dfc_verify_drafts", good, dfc.OK, n_requests=0)
    # groups of 4096 values: 2^24 - 1 of all rows, the drafter's too, and of all requests
    for change in (dict(rows=1 << 24), dict(rows=1 << 20, vocab=65536 + 1), dict(vocab=1 << 30, n_requests=64, rows=64),
                   dict(rows=1 << 23, draft_logits_dev=256)):
        refused("dfc_verify_drafts", good, dfc.EUNSUPPORTED, **dict(dict(logits_stride=1 << 30, draft_stride=1 << 30), **change))
    logits = torch.zeros(5, 1000)
    assert dfc.verify_drafts_workspace(logits, torch.zeros(3, dtype=torch.int32)) == size.value
    assert dfc.verify_drafts_workspace(logits, torch.zeros(3, dtype=torch.int32), logits) == both


def test_sinks_are_refused_past_31_bits():
    f = dfc.library().dfc_paged_attention_sinks
    f.argtypes = [PTR, U32, PTR]
    assert f(None, 4, None) == dfc.EINVAL


def calls():
    """Every new call, all of it on the CPU, and the tensors that it may be
    asked a gradient of."""
    i, c, table = torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int64), torch.zeros(1, 4).int()
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    cache = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    cu, z = torch.zeros(2).int(), torch.zeros(1, 5)
    return [
        (lambda: dfc.paged_release(i, i, table, i, c, i, 16), []),
        (lambda: dfc.paged_fork(i, i, table, i, c, i, 16), []),
        (lambda: dfc.paged_compact(i, table, i, c, i, 16), []),
        (lambda a=cache: dfc.paged_copy([(a, a)], i, i), []),
        (lambda a=z, b=z, u=z[0, :1], t=z[0, :1]: dfc.verify_drafts(a, cu, c[:1], u, draft_logits=b, temperature=t),
         [z, z, z[0, :1], z[0, :1]]),
        (lambda q=x, w=x[0, 0]: dfc.paged_append(x, x, cache, cache, c[:1], q=q, q_norm=w, k_norm=w), []),
        (lambda q=x: dfc.paged_attention(q, cache, cache, table, cu, i, window=3, sinks=2), [x]),
    ]


def test_tensors_off_the_device_are_refused():
    for call, _ in calls():
        with pytest.raises(TypeError, match="device"):
            call()


def test_gradients_are_refused():
    # (the device is asked of the main tensor first, the gradient before)
    for call, args in calls():
        if not args:
            continue
        wants = [a.clone() for a in args]
        wants[0].requires_grad_()
        with pytest.raises(ValueError, match="gradient"):
            call(*wants)
        with torch.no_grad(), pytest.raises(TypeError, match="device"):
            call(*wants)
