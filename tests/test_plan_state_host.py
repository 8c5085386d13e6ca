"""How the layer plans order calls that share their memory (csrc/plan_state.h),
compiled here against a stand-in for the CUDA runtime that writes down waits
and records with the identity of the stream."""

import os
import shutil
import subprocess

import pytest

from gemm_matmulplan_broadcast_gb300.build import CSRC, INCLUDE

HERE = os.path.dirname(os.path.abspath(__file__))


def run(tmp_path, body):
    if not shutil.which("g++"):
        pytest.skip("no g++")
    src = tmp_path / "t.cpp"
    src.write_text('#include "plan_state.h"\nint main() {\n    olc::PlanState p;\n    p.init();\n%s\n    p.destroy();\n'
                   '    std::puts(fake::log.c_str());\n}\n' % body)
    exe = str(tmp_path / "t")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-Wno-misleading-indentation", "-I", os.path.join(HERE, "fake_cuda"), "-I", CSRC, "-I", INCLUDE,
                    str(src), "-o", exe], check=True)
    return subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()


CALL = "p.before_use(%s); p.after_use(%s);"


def test_one_stream_does_not_wait_for_itself(tmp_path):
    log = run(tmp_path, "FakeStream a{7, false};" + 3 * (CALL % ("&a", "&a")))
    assert log == ["record7"] * 3


def test_another_stream_waits(tmp_path):
    log = run(tmp_path, "FakeStream a{7, false}, b{8, false};" + CALL % ("&a", "&a") + CALL % ("&b", "&b") + CALL % ("&a", "&a"))
    assert log == ["record7", "wait8", "record8", "wait7", "record7"]


def test_the_default_streams_of_two_threads_are_two_streams(tmp_path):
    one = CALL % ("fake::per_thread", "fake::per_thread")
    log = run(tmp_path, one + "fake::thread_stream_id = 1001;" + one)
    assert log == ["record1000", "wait1001", "record1001"]


def test_a_handle_that_names_a_new_stream_waits_for_the_old_one(tmp_path):
    log = run(tmp_path, "FakeStream a{7, false};" + CALL % ("&a", "&a") + "a.id = 9;" + CALL % ("&a", "&a"))
    assert log == ["record7", "wait9", "record9"]


def test_captures_are_left_alone(tmp_path):
    log = run(tmp_path, "FakeStream a{7, false}, b{8, true};" + CALL % ("&a", "&a") +
              "if (p.before_use(&b) || p.after_use(&b)) return 1;" + CALL % ("&a", "&a"))
    assert log == ["record7", "record7"]


def test_every_plan_with_memory_follows_this_order():
    # the matrix plans hold the same order; nobody keeps a handle to compare
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        if name == "api.cpp":
            assert "StreamOrder order;" in text and "order." in text
        assert "state_stream" not in text and "stream == s" not in text, name


def test_what_went_ahead_of_a_failure_is_recorded(tmp_path):
    log = run(tmp_path, "FakeStream a{7, false}, b{8, false};"
              "const cudaError_t e = p.use(&a, [] { fake::log += \"work \"; return cudaErrorLaunchFailure; });"
              "if (e != cudaErrorLaunchFailure) return 1;"
              "if (p.use(&b, [] { fake::log += \"work \"; return cudaSuccess; })) return 1;")
    assert log == ["work", "record7", "wait8", "work", "record8"]


def test_plans_enqueue_under_the_order_alone():
    # no call notes its use by hand, where an early return could leave it out
    for name in sorted(os.listdir(CSRC)):
        if name != "stream_order.h":
            with open(os.path.join(CSRC, name)) as f:
                text = f.read()
            assert "before_use(" not in text and "after_use(" not in text, name


def test_an_allocation_that_fails_says_why_and_keeps_what_is_there(tmp_path):
    log = run(tmp_path, "if (p.ensure(100) != OLC_OK) return 1;"
              "void* const before = p.memory;"
              "fake::malloc_result = cudaErrorMemoryAllocation;"
              "if (p.ensure(200) != OLC_ERR_OOM) return 1;"
              # refused for another reason: a capture, say
              "fake::malloc_result = cudaErrorLaunchFailure;"
              "if (p.ensure(200) != OLC_ERR_CUDA) return 1;"
              "if (p.memory != before || p.bytes != 100 || p.earlier) return 1;"
              "fake::malloc_result = cudaSuccess;"
              "if (p.ensure(200) != OLC_OK || p.bytes != 200 || !p.earlier) return 1;")
    assert log == []
