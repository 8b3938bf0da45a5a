"""The paged cache's entry points where no GPU is needed: the workspace's size
through the C ABI, and the Python binding's refusals."""
import ctypes
import os
import subprocess

import pytest

import lossless_entropy_coded_dfc_amd as dfc

torch = pytest.importorskip("torch")
U32, U64, I64, PTR = ctypes.c_uint32, ctypes.c_uint64, ctypes.c_int64, ctypes.c_void_p


class Cache(ctypes.Structure):
    _fields_ = [("k_dev", PTR), ("v_dev", PTR), ("k_stride", I64 * 3), ("v_stride", I64 * 3), ("n_pages", U32),
                ("page_size", U32), ("kv_heads", U32), ("head_dim", U32), ("dtype", U32)]


class Attention(ctypes.Structure):
    _fields_ = [("cache", Cache), ("heads", U32), ("n_requests", U32), ("max_pages", U32), ("max_q_len", U32),
                ("tokens", U64), ("q_dev", PTR), ("out_dev", PTR), ("q_stride", I64 * 2), ("out_stride", I64 * 2),
                ("lse_dev", PTR), ("block_table", PTR), ("table_stride", I64), ("cu_q", PTR), ("seq_lens", PTR),
                ("scale", ctypes.c_float), ("causal", U32), ("window", U32), ("workspace_dev", PTR),
                ("workspace_bytes", U64), ("status_dev", PTR)]


@pytest.mark.parametrize("name,mirror", [("dfc_paged_cache", Cache), ("dfc_attention_args", Attention)])
def test_layout(name, mirror, tmp_path):
    # the structures above against the C compiler's
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


def test_one_workspace_serves_every_window_and_layout():
    # The kernel's shape follows the window and the layouts; the bytes a call
    # asks for are a matter of the sizes alone
    lib = dfc.library()
    lib.dfc_paged_attention_workspace.argtypes = [ctypes.POINTER(Attention), ctypes.POINTER(U64)]
    lib.dfc_paged_attention.argtypes = [ctypes.POINTER(Attention), PTR]

    def args(window, v_stride, dim, heads, n, tokens, width, hint):
        kv = 8
        plain = 16 * kv * dim, kv * dim, dim
        cache = Cache(256, 256, (I64 * 3)(*plain), (I64 * 3)(*v_stride), 4096, 16, kv, dim, 0)
        rows = (I64 * 2)(heads * dim, dim)
        return Attention(cache, heads, n, width, hint, tokens, 256, 256, rows, rows, None, 256, width, 256, 256, 1.0, 1,
                         window, 256, 0, None)

    def need(a):
        out = U64()
        assert lib.dfc_paged_attention_workspace(a, ctypes.byref(out)) == 0
        return out.value

    for dim, heads, n, tokens, width, hint in [(128, 32, 1, 2048, 128, 0), (128, 32, 1, 513, 2032, 513),
                                               (64, 32, 4, 1900, 400, 1900), (128, 32, 16, 680, 2048, 333),
                                               (256, 16, 2, 700, 1000, 0), (80, 8, 3, 300, 9, 0), (128, 32, 64, 64, 512, 1)]:
        sizes = dim, heads, n, tokens, width, hint
        plain = 16 * 8 * dim, 8 * dim, dim
        most = need(args(0, plain, *sizes))
        for window in (0, 1, 64, 777, 5000):
            for layout in (plain, (16 * 8 * dim, dim, 16 * dim)):
                a = args(window, layout, *sizes)
                assert need(a) == most, (sizes, window, layout)
                # no bytes given: refused before anything is launched
                assert lib.dfc_paged_attention(a, None) == dfc.ESIZE, (sizes, window, layout)


def test_refusals_without_a_device():
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    q, i, table = torch.zeros(1, 4, 64, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32), torch.zeros(1, 4).int()
    for call in (lambda: dfc.paged_attention(q, k, k, table, torch.zeros(2).int(), i),
                 lambda: dfc.paged_append(q[:, :2], q[:, :2], k, k, i.long()),
                 lambda: dfc.paged_plan(i, i, table, i, torch.zeros(2).long(), 16, 1),
                 lambda: dfc.paged_attention_workspace(q, k, k, table, i, i),
                 lambda: dfc.paged_attention(None, k, k, table, i, i),
                 lambda: dfc.paged_plan(i, i, table.tolist(), i, i, 16, 1)):
        with pytest.raises(TypeError):
            call()


def test_tensors_that_require_a_gradient_are_refused():
    # there is no backward pass; on the CPU the next refusal is the device's
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    i, table, cu = torch.zeros(1, dtype=torch.int32), torch.zeros(1, 4).int(), torch.zeros(2).int()

    def attention(q, kc, vc):
        dfc.paged_attention(q, kc, vc, table, cu, i)

    def append(kk, vv, kc, vc, q=None, rotary=None):
        dfc.paged_append(kk, vv, kc, vc, i.long(), q=q, positions=i, rotary=rotary)

    for call, args in ((attention, [x, k, k]), (append, [x, x, k, k])):
        with pytest.raises(TypeError, match="device"):
            call(*args)
        for at in range(len(args) if call is append else 1):
            wants = list(args)
            wants[at] = args[at].clone().requires_grad_()
            with pytest.raises(ValueError, match="gradient"):
                call(*wants)
            with torch.no_grad(), pytest.raises(TypeError, match="device"):
                call(*wants)
