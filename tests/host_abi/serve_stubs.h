// State of the serving launchers' stand-ins.
#pragma once
extern int g_cus;  // what device_cus() reports
