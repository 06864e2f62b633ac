"""The give-up paths of the norm's and the recurrence's rings, on the host: every
copy in flight is waited for again, the one whose wait ran out among them."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_copy_in_flight_is_waited_for(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path / "ring_order")
    csrc = os.path.join(ROOT, "selective_state_space_mss_b200", "csrc")
    build = subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I", csrc, os.path.join(ROOT, "tests", "ring_order.cpp"),
                            "-o", exe], capture_output=True, text=True)
    assert build.returncode == 0, build.stderr
    run = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0 and run.stdout.strip() == "ok", run.stdout + run.stderr


def test_the_self_test_is_a_setting_of_the_thread():
    """Also what a call refuses comes first: no launch, no device."""
    import threading

    import selective_state_space_mss_b200 as mss
    from selective_state_space_mss_b200 import build as mss_build

    mss_build.build()
    seen = []
    assert mss.selftest_timeout(True) is False and mss.selftest_timeout(True) is True
    t = threading.Thread(target=lambda: seen.append(mss.selftest_timeout(False)))
    t.start()
    t.join()
    assert seen == [False]
    assert mss.selftest_timeout(False) is True and mss.selftest_timeout(False) is False
