"""What the compiled way into the library does when the library throws, or when Python ends under a call: its own code, compiled
around stand-ins for the library's entries, since every real call needs a GPU."""
import subprocess
import sys

import pytest

STAND_INS = r"""
#include "%s"

#include <new>
#include <unistd.h>

namespace {
PyObject* py_throws(PyObject* const*, Py_ssize_t) {
  return call([]() -> pq_status { throw std::bad_alloc(); });
}
PyObject* py_throws_before(PyObject* const*, Py_ssize_t) { throw std::bad_alloc(); }
PyObject* py_answers(PyObject* const*, Py_ssize_t) {
  return call([]() -> pq_status { return PQ_ERR_INVALID_ARG; });
}
PyObject* py_waits(PyObject* const*, Py_ssize_t) {
  return call([]() -> pq_status { usleep(300000); return PQ_OK; });
}
PyMethodDef stand_ins[] = {PQ_METHOD(throws), PQ_METHOD(throws_before), PQ_METHOD(answers), PQ_METHOD(waits), {nullptr, nullptr, 0, nullptr}};
PyModuleDef stand_in_module = {PyModuleDef_HEAD_INIT, "standins", "", -1, stand_ins, nullptr, nullptr, nullptr, nullptr};
}  // namespace

PyMODINIT_FUNC PyInit_standins() { return PyModule_Create(&stand_in_module); }
"""


@pytest.fixture(scope="module")
def folder(tmp_path_factory):
    from rotation_int4_w4a4_b200 import build
    d = tmp_path_factory.mktemp("standins")
    (d / "standins.cpp").write_text(STAND_INS % build.CALL_SOURCE)
    cmd = build._call_command(str(d / "standins.cpp"), str(d / "standins.so"))
    cmd[cmd.index("-O2")] = "-O1"
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    return d


def python(folder, code):
    res = subprocess.run([sys.executable, "-c", "import torch, sys\nsys.path.insert(0, sys.argv[1])\nimport standins as s\n" + code, str(folder)],
                         capture_output=True, text=True, timeout=120)
    return res.returncode, res.stdout, res.stderr


def test_an_exception_of_the_library_is_raised_in_python(folder):
    """Not -1, which says that the call has had no effect and may be made again; and with the interpreter's lock in hand."""
    code = """
for _ in range(3):
    try:
        print("returned", s.throws())
    except RuntimeError as e:
        print("raised", e)
print("then", s.answers())
"""
    rc, out, err = python(folder, code)
    assert rc == 0, (rc, out, err)
    lines = out.split("\n")
    assert all(x.startswith("raised") and "exception" in x for x in lines[:3]) and lines[3].startswith("then") and int(lines[3][5:]) > 0


def test_an_exception_before_the_library_is_a_call_not_taken(folder):
    assert python(folder, "print(s.throws_before(), s.throws_before())")[:2] == (0, "-1 -1\n")


def test_python_may_end_while_a_call_runs(folder):
    """A daemon thread's call outlasts the interpreter: the thread ends where it asks for the lock, by an unwinding that nothing may
    hold up (a handler that swallows it goes on without the lock)."""
    code = """
import threading, time
threading.Thread(target=s.waits, daemon=True).start()
time.sleep(0.1)
"""
    rc, out, err = python(folder, code)
    assert rc == 0, (rc, out, err)
