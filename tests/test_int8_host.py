"""8-bit serving products on a host without a GPU: exports, argument checks
before any CUDA call, host fault injection, the binding's refusals."""
import json
import os
import re
import subprocess
import sys

import numpy as np
import pytest
import torch

from tests import _int8_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # 16-byte aligned, never dereferenced: validation fails first
ENTRY_POINTS = ["wq_linear_w8a8", "wq_linear_w8a8_grouped", "wq_quantize_tokens"]


@pytest.fixture(scope="module")
def b():
    from w4a16_bit_gemm_b200 import build
    build.build()
    from w4a16_bit_gemm_b200 import binding
    return binding


def test_header_declares_what_the_library_exports(b):
    src = open(os.path.join(ROOT, "include", "wq_int8.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    assert sorted(set(re.findall(r"\b(wq_[a-z0-9_]+)\s*\(", src))) == ENTRY_POINTS
    for n in ENTRY_POINTS:
        assert hasattr(b.lib, n), n
    assert "WQ_DEVFLAG_INDEX 0x8u" in src and b.WQ_DEVFLAG_INDEX == 0x8


@pytest.mark.parametrize("case", [
    dict(X=None), dict(X=FAKE + 8), dict(Xq=None), dict(Xq=FAKE + 4), dict(xs=None), dict(xs=FAKE + 2),
    dict(rows=FAKE + 2, R=4), dict(R=3), dict(T=-1, R=-1), dict(d_in=0), dict(d_in=48), dict(d_in=131072),
    dict(smooth=FAKE + 1), dict(T=1 << 31, R=1 << 31), dict(rows=FAKE, R=-1),
])
def test_quantize_tokens_rejects(b, case):
    a = dict(X=FAKE, T=4, d_in=256, rows=None, R=4, smooth=None, Xq=FAKE, xs=FAKE)
    a.update(case)
    assert b.lib.wq_quantize_tokens(a["X"], a["T"], a["d_in"], a["rows"], a["R"], a["smooth"], a["Xq"], a["xs"],
                                    None) == 1


PRODUCT = dict(Xq=FAKE, xs=FAKE, R=4, q=FAKE, s=FAKE, N=64, K=256, Y=FAKE, ydt=0)
BAD_PRODUCTS = [
    dict(Xq=None), dict(Xq=FAKE + 8), dict(xs=None), dict(xs=FAKE + 2), dict(R=-1), dict(R=1 << 31), dict(q=None),
    dict(q=FAKE + 4), dict(s=None), dict(s=FAKE + 1), dict(N=0), dict(N=1 << 31), dict(K=0), dict(K=100),
    dict(K=131072), dict(Y=None), dict(Y=FAKE + 8), dict(ydt=2),
]


@pytest.mark.parametrize("case", BAD_PRODUCTS)
def test_linear_w8a8_rejects(b, case):
    a = dict(PRODUCT, **case)
    assert b.lib.wq_linear_w8a8(a["Xq"], a["xs"], a["R"], a["q"], a["s"], a["N"], a["K"], a["Y"], a["ydt"], None) == 1


@pytest.mark.parametrize("case", BAD_PRODUCTS + [dict(off=None), dict(off=FAKE + 2), dict(E=0), dict(E=1000, N=1 << 22)])
def test_linear_w8a8_grouped_rejects(b, case):
    a = dict(PRODUCT, off=FAKE, E=8)
    a.update(case)
    assert b.lib.wq_linear_w8a8_grouped(a["Xq"], a["xs"], a["R"], a["off"], a["E"], a["q"], a["s"], a["N"], a["K"],
                                        a["Y"], a["ydt"], None) == 1


def test_too_many_experts_is_unsupported(b):
    assert b.lib.wq_linear_w8a8_grouped(FAKE, FAKE, 4, FAKE, 1025, FAKE, FAKE, 64, 256, FAKE, 0, None) == 2


_INJECT = r'''
import json, sys
sys.path.insert(0, sys.argv[1])
from w4a16_bit_gemm_b200 import binding
lib, F, out = binding.lib, 0x10000, {}
def call(name, *args):
    before = lib.wq_fault_injections()
    st = getattr(lib, name)(*args)
    out[name] = [st, lib.wq_fault_injections() - before]
call("wq_quantize_tokens", F, 4, 256, None, 4, None, F, F, None)
call("wq_linear_w8a8", F, F, 4, F, F, 64, 256, F, 0, None)
call("wq_linear_w8a8_grouped", F, F, 4, F, 8, F, F, 64, 256, F, 0, None)
before = lib.wq_fault_injections()
out["invalid"] = [lib.wq_linear_w8a8(None, F, 4, F, F, 64, 256, F, 0, None), lib.wq_fault_injections() - before]
print(json.dumps(out))
'''


@pytest.mark.parametrize("mode", ["launch", "alloc"])
def test_injected_host_faults_fail_each_call_once(b, mode):
    env = dict(os.environ, WQ_FAULT_INJECT=mode, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-c", _INJECT, ROOT], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    out = json.loads(r.stdout.strip().splitlines()[-1])
    for name in ENTRY_POINTS:
        assert out[name] == [3, 1], (name, out[name])
    assert out["invalid"] == [1, 0]


def test_binding_refuses_cpu_tensors(b):
    X = torch.zeros(4, 256, dtype=torch.bfloat16)
    q = torch.zeros(64, 64, dtype=torch.int32)
    p = b.PackedLinearW8(q, torch.ones(64, 1, dtype=torch.float16), 64, 256, 256)
    pe = b.PackedExpertsW8(q.view(2, 32, 64), torch.ones(2, 32, dtype=torch.float16))
    off = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: b.quantize_tokens(X), lambda: b.linear_w8a8(X, p), lambda: b.linear_w8a8_grouped(X, pe, off),
                 lambda: b.quantize_w8_experts(torch.zeros(2, 32, 256, dtype=torch.bfloat16))):
        with pytest.raises(ValueError, match="no CPU fallback"):
            call()


# The tests' own plain definition, against torch and closed forms.

def test_reference_quantizer():
    x = torch.tensor([[127.0, -63.5, 0.5, 1.5, 2.5, 0.0, -0.5, 1.0]]).to(torch.bfloat16)
    q, s, bad = ref.quantize_tokens(x)
    assert s[0] == 1.0 and not bad
    assert q[0].tolist() == [127, -64, 0, 2, 2, 0, 0, 1]  # ties to even; -63.5 -> -64
    q, s, bad = ref.quantize_tokens(torch.zeros(1, 8).to(torch.bfloat16))
    assert s[0] == 1.0 and not q.any()
    x = torch.tensor([[float("nan"), float("inf"), -float("inf"), 2.0]]).to(torch.bfloat16)
    q, s, bad = ref.quantize_tokens(x)
    assert bad and q[0].tolist() == [0, 127, -127, 127] and s[0] == np.float32(2) / np.float32(127)


def test_reference_product():
    rng = np.random.default_rng(1)
    xq, wq = rng.integers(-128, 128, (5, 96)), rng.integers(-128, 128, (7, 96))
    assert np.array_equal(ref.sums(xq, wq), xq @ wq.T)
    y, y64 = ref.product(xq, np.full(5, 0.5), wq, np.full(7, 0.25))  # powers of two: no rounding
    assert np.array_equal(y64, (xq @ wq.T) / 8) and np.array_equal(y, y64)


def test_reference_words_are_the_w8_layout():
    import oracle
    W = torch.randn(5, 64, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    oq, _, _, codes = oracle.quantize_pack8(W.view(torch.int16).numpy().view(np.uint16), 64)
    assert np.array_equal(ref.words(codes.astype(np.int8)).numpy().view(np.uint32), oq)


# Orders inside the kernels that no run can be asked to show: what goes wrong
# without them may not end.

def kernel_source(name, start):
    """The body of the kernel that `start` opens, without comments, in one line."""
    src = open(os.path.join(ROOT, "w4a16_bit_gemm_b200", "csrc", name)).read()
    src = re.sub(r"//[^\n]*", "", src)
    body = src[src.index(start):]
    return " ".join(body[:body.index("\n}\n")].split())


def in_order(body, *parts):
    at = [0]
    for p in parts:
        assert p in body[at[-1]:], (p, "missing, or before", parts)
        at.append(body.index(p, at[-1]) + len(p))


def test_pair_kernel_allocates_once_both_ctas_run():
    """The allocation of a CTA pair waits without a limit for a warp of each: a
    barrier of the cluster comes first, and another before the first use and
    before the memory is given back."""
    body = kernel_source("w8a8_pair.cu", "w8a8_pair_kernel(")
    barrier = "cluster_arrive(); cluster_wait();"
    in_order(body, barrier, "tcgen05.alloc", barrier, "tc_mma_i8_pair", barrier, "tcgen05.dealloc")


def test_pair_kernel_never_runs_beside_another():
    """Neither started early nor a starter of others: no wait for an earlier
    kernel can then hold an SM, or tensor memory, that the pair needs."""
    src = open(os.path.join(ROOT, "w4a16_bit_gemm_b200", "csrc", "w8a8_pair.cu")).read()
    src = re.sub(r"//[^\n]*", "", src)
    for word in ("pdl_launch_dependents", "pdl_wait_prior", "griddepcontrol", "ProgrammaticStreamSerialization"):
        assert word not in src, word


def test_pair_kernel_waits_for_its_last_arrivals():
    """Both CTAs stay until the last commits have arrived on their own barriers,
    the leader also until both CTAs' last copies have."""
    body = kernel_source("w8a8_pair.cu", "w8a8_pair_kernel(")
    loop = body[body.index("for (int j = max(0, it - kStages); j < it; ++j) {"):]
    loop = loop[:loop.index("__syncwarp();")]
    assert re.search(r"if \(rank == 0\) mbar_wait\w*\(&bar\.full\[.*?; mbar_wait\w*\(&bar\.empty\[", loop), loop


def test_partials_of_other_ctas_are_acquired_from_the_cluster():
    """st.async signals at cluster scope: so does the wait ahead of the reads."""
    body = kernel_source("w8a8_stream.cu", "w8a8_stream_kernel(")
    in_order(body, "st_async_v4(", "mbar_wait_cluster(&bar.recv,", "recv[(s * pitch + g) * kCh + ch]")
    assert "mbar_wait(&bar.recv" not in body


def test_pair_kernel_acquires_from_the_cluster():
    """Every barrier but the leader's own last one is completed by the other
    CTA's copies, commits or arrivals."""
    body = kernel_source("w8a8_pair.cu", "w8a8_pair_kernel(")
    assert re.findall(r"mbar_wait\((&bar\.\w+)", body) == ["&bar.drain"]
    assert len(re.findall(r"mbar_wait_cluster\(&bar\.(?:full|empty|acc_full|acc_empty)\[", body)) == 6


def test_stream_kernel_holds_no_tensor_memory_before_the_work_ahead_with_experts():
    """With experts: the wait, the allocation, and only then the next kernel's
    start.  With one matrix: the allocation, then the next kernel's start."""
    body = kernel_source("w8a8_stream.cu", "w8a8_stream_kernel(")
    in_order(body, "if (a.offsets) pdl_wait_prior();", "tmem_alloc(", "build_tiles(", "pdl_launch_dependents();",
             "tmem_dealloc(")
    assert body.count("tmem_alloc(") == 1 and body.count("pdl_launch_dependents();") == 1
