// tc_common.cuh for the paged entries' translation unit: the device variables it defines (status
// word, wait limit, test hook) get names of their own, since each unit has its own copy.
// infini_attn_device_status and the test hooks see to both.
#pragma once

#define g_wait_status g_paged_wait_status
#define g_spin_limit g_paged_spin_limit
#define g_test_withhold g_paged_test_withhold
#include "tc_common.cuh"
#undef g_wait_status
#undef g_spin_limit
#undef g_test_withhold
